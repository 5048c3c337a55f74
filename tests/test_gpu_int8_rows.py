"""Every row and entry of the INT8 product, where the row tiles pass a full super-group of the
persistent form, whose XCDs take every eighth of them."""
import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def m():
    from mask_only_logits_amd import mosaic
    return mosaic


def _codes(seed, n, d):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-128, 128, (n, d), generator=g, dtype=torch.int8)
    return q.to(DEV), (torch.rand(n, generator=g) * 0.02 + 1e-3).to(DEV)


@pytest.mark.parametrize("M,V,d", [(8300, 400, 128), (8300, 400, 640), (8300, 400, 400), (16484, 600, 128),
                                   (16484, 600, 304), (33000, 300, 128), (9000, 2500, 256), (1100, 25600, 128),
                                   (1300, 2501, 127), (600, 30000, 400)])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_int8_every_row(m, M, V, d, out_dtype):
    hq, hs = _codes(M, M, d)
    wq, ws = _codes(V, V, d)
    out = torch.full((M + 1, V), 7.0, dtype=out_dtype, device=DEV)
    m.mosaic_quantized_logits(hq, hs, wq, ws, out=out)
    wt = wq.double().t().contiguous()
    for r in range(0, M, 4096):
        rows = slice(r, min(M, r + 4096))
        want = torch.mm(hq[rows].double(), wt) * hs[rows].double()[:, None] * ws.double()
        # the sum's conversion and two products: three roundings
        tol = want.abs() * (plain64.HALF[out_dtype] + 4 * plain64.U32) + plain64.TINY
        bad = (out[rows].double() - want).abs() > tol
        assert not bool(bad.any()), (r, bad.nonzero()[:4].tolist())
    assert bool((out[M] == 7).all())
    # 32 rows at a time: another form, the same bits
    for r in range(0, M, 32):
        part = m.mosaic_quantized_logits(hq[r:r + 32], hs[r:r + 32], wq, ws, out_dtype=out_dtype)
        assert torch.equal(part, out[r:min(M, r + 32)]), r
