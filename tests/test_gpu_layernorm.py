"""Layer norm with residual addition and its gradient against 64-bit arithmetic."""
import math

import pytest
import torch

import head64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
WIDTHS = [1, 2, 7, 8, 31, 64, 65, 127, 128, 190, 192, 255, 256, 300, 384, 511, 512, 520, 768, 1000, 1021, 1024, 1400, 1536,
          2047, 2048, 2500, 2560, 2600, 4096, 4097, 6000, 6144, 8191, 8192, 10000, 16384, 16385, 20001]


@pytest.fixture(scope="module")
def m():
    from mask_only_logits_amd import mosaic
    return mosaic


def _draw(seed, n, d, dtype, far=0.5):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g, device=DEV)
    return ((normal(n, d) * torch.exp(0.7 * normal(d)) + far * normal(d)).to(dtype), normal(n, d).to(dtype),
            (1 + 0.2 * normal(d)), 0.2 * normal(d), (1e-2 * normal(n, d)).to(dtype), (1e-2 * normal(n, d)).to(dtype))


def _strided(t, extra, shift):
    """The same values in rows of another stride, from another address on."""
    n, d = t.shape
    big = torch.full((n * (d + extra) + shift,), 7.0, dtype=t.dtype, device=t.device)
    v = big[shift:].view(n, d + extra)[:, :d]
    v.copy_(t)
    return v, big


@pytest.mark.parametrize("dtype,gt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("d", WIDTHS)
def test_widths(m, d, dtype, gt):
    n = 37
    x, r, gain, bias, dy, ds = _draw(d, n, d, dtype)
    gain, bias = gain.to(gt), bias.to(gt)
    s, y, st = m.mosaic_add_layernorm(x, gain, bias, residual=r, store_sum=True, with_stats=True)
    head64.check_layernorm(x, r, gain, bias, 1e-5, None, s, y, st, f"{d}")
    _, y, st = m.mosaic_add_layernorm(x, gain, bias, with_stats=True)
    head64.check_layernorm(x, None, gain, bias, 1e-5, None, None, y, st, f"{d} alone")
    dx, dg, db = m.mosaic_layernorm_grad(dy, x, st, gain, grad_sum=ds)
    head64.check_layernorm_grad(dy, x, st, gain, None, ds, dx, dg, db, f"{d}")
    dx, dg, db = m.mosaic_layernorm_grad(dy, x, st, gain)
    head64.check_layernorm_grad(dy, x, st, gain, None, None, dx, dg, db, f"{d} alone")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,d", [(1, 1), (1, 4096), (2, 64), (3, 129), (255, 64), (1025, 192), (5000, 512), (4099, 1021),
                                 (3001, 4096), (1500, 2304), (700, 8192), (300, 12288)])
def test_row_counts(m, n, d, dtype):
    x, r, gain, bias, dy, ds = _draw(n + d, n, d, dtype)
    s, y, st = m.mosaic_add_layernorm(x, gain, bias, residual=r, store_sum=True, with_stats=True)
    head64.check_layernorm(x, r, gain, bias, 1e-5, None, s, y, st)
    dx, dg, db = m.mosaic_layernorm_grad(dy, s, st, gain, grad_sum=ds)
    head64.check_layernorm_grad(dy, s, st, gain, None, ds, dx, dg, db)
    again = m.mosaic_layernorm_grad(dy, s, st, gain, grad_sum=ds)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dg, db)))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,extra,shift", [(64, 1, 0), (100, 3, 1), (1021, 7, 3), (4096, 8, 1), (4090, 0, 5), (17000, 1, 1)])
def test_strides_and_addresses(m, d, extra, shift, dtype):
    n = 19
    x, r, gain, bias, dy, ds = _draw(d, n, d, dtype)
    xs, _ = _strided(x, extra, shift)
    rs, _ = _strided(r, extra + 2, shift + 1)
    so, big = _strided(torch.zeros_like(x), extra + 1, shift)
    so.fill_(0)
    s, y, st = m.mosaic_add_layernorm(xs, gain, bias, residual=rs, sum_out=so, with_stats=True)
    head64.check_layernorm(x, r, gain, bias, 1e-5, None, s, y, st)
    assert bool((big[:shift] == 7).all()) and bool((big[shift:].view(n, -1)[:, d:] == 7).all())
    dys, _ = _strided(dy, extra, shift)
    dss, _ = _strided(ds, extra + 3, shift + 2)
    dxs, big = _strided(torch.zeros_like(x), extra + 1, shift)
    _, dg, db = m.mosaic_layernorm_grad(dys, so, st, gain, grad_sum=dss, grad_x=dxs)
    head64.check_layernorm_grad(dy, s, st, gain, None, ds, dxs, dg, db)
    assert bool((big[:shift] == 7).all()) and bool((big[shift:].view(n, -1)[:, d:] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [96, 1021, 4096, 17000])
def test_in_place(m, d, dtype):
    n = 50
    x, r, gain, bias, dy, ds = _draw(d + 1, n, d, dtype)
    s, y, st = m.mosaic_add_layernorm(x, gain, bias, residual=r, store_sum=True, with_stats=True)
    for into in (x, r):
        a, b = x.clone(), r.clone()
        dst = a if into is x else b
        _, y2, st2 = m.mosaic_add_layernorm(a, gain, bias, residual=b, sum_out=dst, with_stats=True)
        assert torch.equal(dst, s) and torch.equal(y, y2) and torch.equal(st, st2)
    want = m.mosaic_layernorm_grad(dy, s, st, gain, grad_sum=ds)
    for k in range(3):
        t = [dy.clone(), ds.clone(), s.clone()]
        got = m.mosaic_layernorm_grad(t[0], t[2], st, gain, grad_sum=t[1], grad_x=t[k])
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 1000, 4096, 16500])
def test_gathered_rows_with_repeats_and_a_count(m, d, dtype):
    n, L = 30, 80
    x, r, gain, bias, _, _ = _draw(d + 2, L, d, dtype)
    _, _, _, _, dy, ds = _draw(d + 3, n, d, dtype)
    idx = torch.randint(0, L, (n,), generator=torch.Generator().manual_seed(d)).to(torch.int32).to(DEV)
    idx[5] = idx[3]
    s, y, st = m.mosaic_add_layernorm(x, gain, bias, residual=r, row_idx=idx, store_sum=True, with_stats=True)
    head64.check_layernorm(x, r, gain, bias, 1e-5, idx, s, y, st)
    _, y, st = m.mosaic_add_layernorm(x, gain, bias, row_idx=idx, with_stats=True)
    dx, dg, db = m.mosaic_layernorm_grad(dy, x, st, gain, row_idx=idx, grad_sum=ds)
    head64.check_layernorm_grad(dy, x, st, gain, idx, ds, dx, dg, db)
    for c in (-3, 0, 1, 17, n, n + 9):
        k = max(0, min(c, n))
        count = torch.tensor([c], dtype=torch.int32, device=DEV)
        out, stats = torch.full_like(y, 3), torch.full_like(st, 3)
        m.mosaic_add_layernorm(x, gain, bias, row_idx=idx, count=count, out=out, stats=stats)
        assert torch.equal(out[:k], y[:k]) and bool((out[k:] == 3).all())
        assert torch.equal(stats[:k], st[:k]) and bool((stats[k:] == 3).all())
        gx = torch.full_like(dx, 3)
        _, dg, db = m.mosaic_layernorm_grad(dy, x, st, gain, row_idx=idx, grad_sum=ds, count=count, grad_x=gx)
        assert torch.equal(gx[:k], dx[:k]) and bool((gx[k:] == 3).all())
        if k:
            head64.check_layernorm_grad(dy[:k], x, st[:k], gain, idx[:k], None, None, dg, db)
        else:
            assert bool((dg == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 4096, 16500])
def test_row_ids_outside_give_rows_of_nan(m, d, dtype):
    x, _, gain, bias, dy, _ = _draw(d + 4, 6, d, dtype)
    idx = torch.tensor([0, -1, 2, 6, 2 ** 31 - 1, 5], dtype=torch.int32, device=DEV)
    bad = torch.tensor([False, True, False, True, True, False], device=DEV)
    _, y, st = m.mosaic_add_layernorm(x, gain, bias, row_idx=idx, with_stats=True)
    assert bool(torch.isnan(y[bad]).all()) and bool(torch.isfinite(y[~bad]).all()) and bool(torch.isnan(st[bad]).all())
    dx, dg, _ = m.mosaic_layernorm_grad(dy, x, torch.zeros_like(st), gain, row_idx=idx)
    assert bool(torch.isnan(dx[bad]).all()) and bool(torch.isfinite(dx[~bad]).all()) and bool(torch.isnan(dg).all())


@pytest.mark.parametrize("d", [64, 1021, 4096, 16500])
def test_no_rows_no_weights_parts(m, d):
    x, _, gain, bias, dy, _ = _draw(d + 5, 9, d, BF)
    none = x[:0]
    assert m.mosaic_add_layernorm(none, gain, bias)[1].shape == (0, d)
    dx, dg, db = m.mosaic_layernorm_grad(none, none, torch.empty(0, 2, dtype=torch.float64, device=DEV), gain)
    assert dx.shape == (0, d) and bool((dg == 0).all()) and bool((db == 0).all())
    # no gain, no bias, and each output alone
    _, y, st = m.mosaic_add_layernorm(x, with_stats=True)
    head64.check_layernorm(x, None, None, None, 1e-5, None, None, y, st)
    _, y2, _ = m.mosaic_add_layernorm(x, None, bias)
    head64.check_layernorm(x, None, None, bias, 1e-5, None, None, y2, None)
    _, none, st2 = m.mosaic_add_layernorm(x, gain, bias, store_out=False, with_stats=True)
    assert none is None and torch.equal(st, st2)
    whole = m.mosaic_layernorm_grad(dy, x, st, None)
    head64.check_layernorm_grad(dy, x, st, None, None, None, *whole)
    for k in range(3):
        flags = dict(zip(("with_x", "with_gain", "with_bias"), (i == k for i in range(3))))
        part = m.mosaic_layernorm_grad(dy, x, st, None, **flags)
        assert [p is not None for p in part] == [i == k for i in range(3)] and torch.equal(part[k], whole[k])


@pytest.mark.parametrize("d", [5, 64, 1000, 4096, 16500])
def test_values_at_the_edges(m, d):
    g = torch.Generator(device=DEV).manual_seed(d)
    x = torch.randn(8, d, generator=g, device=DEV)
    x[0] = 2.5                                   # constant: y = bias
    x[1] = x[1] * 1e-3 + 4096.0                  # far from zero
    x[2] *= 1e30                                 # squares past fp32
    x[3] *= 1e-30
    x[4, 0] = 1e8                                # an outlier in the place of the shift
    x[5] = 3e38 * torch.sign(x[5])
    x[6, d // 2] = math.inf
    x[7, d // 3] = math.nan
    gain = 1 + 0.2 * torch.randn(d, generator=g, device=DEV)
    bias = torch.randn(d, generator=g, device=DEV)
    _, y, st = m.mosaic_add_layernorm(x, gain, bias, eps=1e-5, with_stats=True)
    head64.check_layernorm(x[:6], None, gain, bias, 1e-5, None, None, y[:6], st[:6])
    assert torch.equal(y[0], bias) and bool(torch.isnan(y[6:]).all())
    dy = torch.randn(8, d, generator=g, device=DEV)
    dx, _, _ = m.mosaic_layernorm_grad(dy[:6], x[:6], st[:6], gain)
    head64.check_layernorm_grad(dy[:6], x[:6], st[:6], gain, None, None, dx)


@pytest.mark.parametrize("d", [48, 1021])
def test_gradient_against_differences(m, d):
    x, _, gain, bias, dy, _ = _draw(d + 6, 3, d, F32)
    _, _, st = m.mosaic_add_layernorm(x, gain, bias, with_stats=True)
    dx, dg, db = m.mosaic_layernorm_grad(dy, x, st, gain)

    def loss(x, g, b):
        u = x - x.mean(1, keepdim=True)
        return (dy.double() * (u / torch.sqrt((u * u).mean(1, keepdim=True) + 1e-5) * g + b)).sum()
    args = [x.double(), gain.double(), bias.double()]
    gen = torch.Generator(device=DEV).manual_seed(1)
    for k, grad in enumerate((dx, dg, db)):
        for _ in range(4):
            v = torch.randn(args[k].shape, generator=gen, device=DEV, dtype=torch.float64)
            h = 1e-4
            up, down = list(args), list(args)
            up[k], down[k] = args[k] + h * v, args[k] - h * v
            # the difference quotient is off by h^2 / 6 of the third derivative, which the deviation's
            # order of 1 keeps near the gradient's size; fp32 results by 100 half steps
            size = float((grad.double() * v).abs().sum()) + float(dy.double().abs().mean())
            assert abs(float((loss(*up) - loss(*down)) / (2 * h)) - float((grad.double() * v).sum())) <= 1e-4 * size


def test_long_rows_of_memory(m):
    # offsets past 2^31 elements: the last rows of a large array
    d, n = 4096, (1 << 31) // 4096 + 3
    x = torch.zeros(n, d, dtype=BF, device=DEV)
    x[-2:] = torch.randn(2, d, generator=torch.Generator().manual_seed(0)).to(BF).to(DEV)
    gain, bias = torch.ones(d, device=DEV), torch.zeros(d, device=DEV)
    _, y, st = m.mosaic_add_layernorm(x, gain, bias, with_stats=True)
    head64.check_layernorm(x[-2:], None, gain, bias, 1e-5, None, None, y[-2:], st[-2:])
    assert bool((y[:4] == 0).all())
    dx, dg, db = m.mosaic_layernorm_grad(x, x, st, gain)
    head64.check_layernorm_grad(x[-2:], x[-2:], st[-2:], gain, None, None, dx[-2:])
    head64.check_layernorm_grad(x[-2:], x[-2:], st[-2:], gain, None, None, None, dg, db)


@pytest.mark.parametrize("d", [40, 190, 500, 700, 1021])
def test_weight_gradients_of_very_many_rows(m, d):
    # more than 128 rows to each group of threads: the sums are taken in runs
    n = 2 ** 30 // d + 7
    g = torch.Generator(device=DEV).manual_seed(d)
    x = torch.randn(n, d, generator=g, device=DEV, dtype=torch.float32).to(BF)
    dy = (1 + torch.rand(n, d, generator=g, device=DEV)).to(BF)     # sums that grow
    _, _, st = m.mosaic_add_layernorm(x, with_stats=True, store_out=False)
    _, dg, db = m.mosaic_layernorm_grad(dy, x, st, with_x=False)
    want_g, want_b = torch.zeros(d, dtype=torch.float64, device=DEV), torch.zeros(d, dtype=torch.float64, device=DEV)
    size_g = torch.zeros_like(want_g)
    for i in range(0, n, 1 << 17):
        k = slice(i, i + (1 << 17))
        t = dy[k].double() * ((x[k].double() - st[k, :1]) * st[k, 1:])
        want_g, want_b, size_g = want_g + t.sum(0), want_b + dy[k].double().sum(0), size_g + t.abs().sum(0)
    # runs of 128 rows in fp32, 4 half steps for a term, one rounding of the result
    assert bool(((dg.double() - want_g).abs() <= 134 * 2.0 ** -24 * size_g).all())
    assert bool(((db.double() - want_b).abs() <= 130 * 2.0 ** -24 * want_b).all())
