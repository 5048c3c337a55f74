"""Layer norm and its gradient on rows whose mean is far larger than their deviation."""
import pytest
import torch

import head64
from plain64 import HALF, TINY, U32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
# widths that leave threads without an element, for each number of threads and chunks that a row takes, and some that do not
WIDTHS = [5, 60, 100, 128, 190, 200, 300, 500, 700, 1000, 1021, 1400, 2000, 2500, 4000, 4096, 6000, 8000, 12000, 16001, 16501,
          20005]


@pytest.fixture(scope="module")
def m():
    from mask_only_logits_amd import mosaic
    return mosaic


def _check_constant_rows(m, d, dtype, eps):
    """Rows of one value, between others.  Their xh is 0, so y is the bias, dx is rho (a - mean(a)) + dsum
    with the tolerance of head64.check_layernorm_grad, and the gain's gradient has nothing of them."""
    g = torch.Generator(device=DEV).manual_seed(d)

    def normal(*s):
        return torch.randn(*s, generator=g, device=DEV)
    x = normal(9, d)
    value = {1: 1.5e36, 2: torch.finfo(dtype).min, 3: 3e38, 5: -2.0 ** 121, 6: 2.0 ** 110, 7: torch.finfo(dtype).max}
    for i, v in value.items():
        x[i] = v
    x = x.to(dtype)
    same = torch.tensor([i in value for i in range(9)], device=DEV)
    gain, bias = 1 + 0.2 * normal(d), normal(d)
    dy, ds = normal(9, d).to(dtype), normal(9, d).to(dtype)
    _, y, st = m.mosaic_add_layernorm(x, gain, bias, eps=eps, with_stats=True)
    head64.check_layernorm(x[~same], None, gain, bias, eps, None, None, y[~same], st[~same], f"{d}")
    rho = float(torch.tensor(eps, dtype=torch.float32).double().rsqrt())
    assert torch.equal(st[same, 0], x[same, 0].double())
    assert bool(((st[same, 1] / rho - 1).abs() <= 2.0 ** -50).all())
    assert torch.equal(y[same], bias.to(dtype).expand(len(value), d))
    for dsum in (None, ds):
        dx, dg, db = m.mosaic_layernorm_grad(dy, x, st, gain, grad_sum=dsum)
        part = None if dsum is None else dsum[~same]
        head64.check_layernorm_grad(dy[~same], x[~same], st[~same], gain, None, part, dx[~same], dg, None, f"{d}")
        assert bool(((db.double() - dy.double().sum(0)).abs() <= 130 * U32 * dy.double().abs().sum(0) + TINY).all())
        a = dy[same].double() * gain.double()
        c1 = a.mean(1, keepdim=True)
        want = rho * (a - c1) + (0.0 if dsum is None else dsum[same].double())
        tol = rho * U32 * (5 * (a.abs() + c1.abs()) + 80 * a.abs().mean(1, keepdim=True))
        tol = tol + want.abs() * (HALF[dtype] + 2 * U32) + TINY
        assert bool(((dx[same].double() - want).abs() <= tol).all()), f"{d}"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", WIDTHS)
def test_constant_rows_far_from_zero(m, d, dtype):
    # mean times rho passes fp32's range
    _check_constant_rows(m, d, dtype, 1e-5)


@pytest.mark.parametrize("eps", [2.0 ** -126, 2.0 ** -124, 2.0 ** -100])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", WIDTHS)
def test_constant_rows_with_the_smallest_eps(m, d, dtype, eps):
    # rho is as large as it can be, 2^63, beside the largest means
    _check_constant_rows(m, d, dtype, eps)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [100, 1021, 4096, 16501])
def test_rows_of_any_deviation(m, d, dtype):
    # either side of 2^60, where rows are scaled, up to the largest values and down to an eps that counts alone
    g = torch.Generator(device=DEV).manual_seed(d)
    scale = torch.tensor([2.0 ** e for e in (-70, -10, 50, 59, 60, 61, 70, 100, 120, 125, 126)], dtype=torch.float64,
                         device=DEV)[:, None]
    unit = 2 * torch.rand(len(scale), d, generator=g, device=DEV, dtype=torch.float64) - 1
    for mean in (0.0, 1.0, -1.5):
        x = ((unit + mean) * scale).to(dtype)
        gain, bias = 1 + 0.2 * torch.randn(d, generator=g, device=DEV), torch.randn(d, generator=g, device=DEV)
        _, y, st = m.mosaic_add_layernorm(x, gain, bias, with_stats=True)
        head64.check_layernorm(x, None, gain, bias, 1e-5, None, None, y, st, f"{d} {mean}")
        for size in (1.0, 2.0 ** 100):   # gradients of rho's size and far above
            dy = (size * torch.randn(len(scale), d, generator=g, device=DEV)).to(dtype)
            dx, _, _ = m.mosaic_layernorm_grad(dy, x, st, gain, with_gain=False, with_bias=False)
            rows = st[:, 1] * size < 2.0 ** 120   # what fp32 holds
            head64.check_layernorm_grad(dy[rows], x[rows], st[rows], gain, None, None, dx[rows], what=f"{d} {mean} {size}")
