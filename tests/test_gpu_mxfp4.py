"""MXFP4 codes, bit for bit, and the head on them against 64-bit arithmetic."""
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


def _normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


def _check_codes(m, x, idx=None, **kw):
    q, s, v = m.mosaic_quantize_rows_mxfp4(x, row_idx=idx, with_values=True, **kw)
    rows = x if idx is None else x[idx.long()]
    wq, ws = head64.mxfp4_codes(rows)
    assert torch.equal(s.cpu(), ws)
    assert torch.equal(q.cpu(), wq)
    want = head64.mxfp4_values(wq, ws, x.shape[1])
    assert v.dtype == x.dtype and torch.equal(torch.nan_to_num(v.cpu().double(), 77.0), torch.nan_to_num(want, 77.0))
    return q, s, v


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,d", [(1, 1), (3, 5), (7, 31), (5, 32), (9, 33), (20, 64), (33, 100), (300, 127), (17, 1040),
                                 (50, 4096), (4099, 96), (2, 20001), (1000, 1021)])
def test_codes(m, n, d, dtype):
    x = (_normal(n + d, n, d) * torch.exp(2 * _normal(d, d))).to(dtype)
    q, s, v = _check_codes(m, x)
    assert bool((head64.mxfp4_values(q, s, 32 * s.shape[1])[:, d:] == 0).all())
    idx = torch.randint(0, n, (n + 3,), generator=torch.Generator().manual_seed(n)).to(torch.int32).to(DEV)
    _check_codes(m, x, idx)
    # values alone, and over the rows themselves
    _, _, only = m.mosaic_quantize_rows_mxfp4(x, store_codes=False, with_values=True)
    y = x.clone()
    m.mosaic_quantize_rows_mxfp4(y, store_codes=False, values=y)
    assert torch.equal(only, v) and torch.equal(y, v)
    again = m.mosaic_quantize_rows_mxfp4(x)
    assert torch.equal(again[0], q) and torch.equal(again[1], s) and again[2] is None


@pytest.mark.parametrize("dtype", [BF, F32])
def test_codes_every_step_and_tie(m, dtype):
    # each representable value, each midpoint and the numbers next to them, at many scales
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])
    near = torch.cat([mids, torch.nextafter(mids, torch.zeros(8)), torch.nextafter(mids, torch.full((8,), 9.0))])
    vals = torch.cat([near, -near, head64.E2M1.float(), -head64.E2M1.float()])
    rows = []
    for e in range(-126, 124, 5):
        for part in vals.split(31):
            row = torch.zeros(32)
            row[:len(part)] = part * 2.0 ** e
            row[31] = 4.0 * 2.0 ** e            # the block's scale
            rows.append(row)
    _check_codes(m, torch.stack(rows).to(dtype).to(DEV))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_codes_edges(m, dtype):
    tiny, top = torch.finfo(dtype).smallest_normal, torch.finfo(dtype).max
    x = torch.zeros(8, 70)
    x[1, 40] = tiny
    x[2, 33:60] = top
    x[3, 5] = math.inf
    x[4, 69] = math.nan
    x[5] = -0.0
    x[6, 0] = 2.0 ** -133                       # a subnormal of both types
    x[7, :32] = torch.linspace(-1, 1, 32) * 2.0 ** -126
    q, s, v = _check_codes(m, x.to(dtype).to(DEV))
    assert s[0, 0] == 0 and s[3, 0] == 255 and s[4, 2] == 255 and bool(torch.isnan(v[3, :32].float()).all())
    bad = torch.tensor([0, -1, 8, 2], dtype=torch.int32, device=DEV)
    q, s, v = m.mosaic_quantize_rows_mxfp4(x.to(dtype).to(DEV), row_idx=bad, with_values=True)
    assert bool((s[1:3] == 255).all()) and bool((q[1:3] == 0).all()) and bool(torch.isnan(v[1:3].float()).all())


SHAPES = [(1, 1, 1), (1, 16, 32), (3, 5, 33), (16, 17, 64), (20, 500, 96), (31, 1000, 1040), (33, 700, 250), (64, 129, 511),
          (65, 640, 512), (77, 1021, 1040), (100, 300, 4000), (128, 512, 768), (129, 1500, 1024), (200, 4100, 544),
          (256, 2048, 2048), (300, 3333, 256), (513, 1031, 1536), (1000, 2500, 320), (20, 30000, 3584), (48, 9000, 1500)]


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,V,d", SHAPES)
def test_logits(m, M, V, d, out):
    h, w = _normal(M + d, M, d), _normal(V + d, V, d) * torch.exp(_normal(V, V, 1))
    hq, hs, _ = m.mosaic_quantize_rows_mxfp4(h)
    wq, ws, _ = m.mosaic_quantize_rows_mxfp4(w.to(BF))
    got = m.mosaic_quantized_logits_mxfp4(hq, hs, wq, ws, out_dtype=out)
    head64.check_mxfp4_logits(got, hq, hs, wq, ws, d, f"{M} x {V} x {d}")
    # a count of rows on the device, and the rows of a smaller call, bit for bit
    k = max(1, M // 3)
    part = m.mosaic_quantized_logits_mxfp4(hq, hs, wq, ws, M=k, out_dtype=out)
    assert torch.equal(part, got[:k])
    for c in (-1, 0, k, M + 1):
        n = max(0, min(c, M))
        to = torch.full_like(got, 3)
        m.mosaic_quantized_logits_mxfp4(hq, hs, wq, ws, count=torch.tensor([c], dtype=torch.int32, device=DEV), out=to)
        assert torch.equal(to[:n], got[:n]) and bool((to[n:] == 3).all())


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("d", [64, 100, 512, 3584])
def test_masked_logits_and_chunks(m, d, out):
    L, M, V = 900, 333, 1003
    H = _normal(d, L, d).to(BF)
    wq, ws, _ = m.mosaic_quantize_rows_mxfp4(_normal(d + 1, V, d))
    idx = torch.randint(0, L, (M,), generator=torch.Generator().manual_seed(d)).to(torch.int32).to(DEV)
    hq, hs, _ = m.mosaic_quantize_rows_mxfp4(H, row_idx=idx)
    want = m.mosaic_quantized_logits_mxfp4(hq, hs, wq, ws, out_dtype=out)
    for C in (0, 1, 20, 64, 100, 332, 333, 1000):
        got = m.mosaic_masked_logits_mxfp4(H, idx, wq, ws, out_dtype=out, chunk_rows=C)
        assert torch.equal(got, want), f"chunks of {C}"
    got = m.mosaic_masked_logits_mxfp4(H.float(), idx, wq, ws, M=50, out_dtype=out)
    assert torch.equal(got, want[:50])


def test_masked_logits_row_ids(m, lib_env):
    H, (wq, ws, _) = _normal(1, 10, 96).to(BF), m.mosaic_quantize_rows_mxfp4(_normal(2, 40, 96))
    idx = torch.tensor([3, 10, -1, 0], dtype=torch.int32, device=DEV)
    got = m.mosaic_masked_logits_mxfp4(H, idx, wq, ws)
    assert bool(torch.isnan(got[1:3]).all()) and bool(torch.isfinite(got[[0, 3]]).all())
    lib_env("MOSAIC_CHECK_IDX", "1")
    with pytest.raises(m.MosaicError):
        m.mosaic_masked_logits_mxfp4(H, idx, wq, ws)


@pytest.mark.parametrize("M", [1, 20, 70, 300])
def test_scales_at_the_edges(m, M):
    # scales that meet in the product's range, and a NaN scale that takes its row or column alone
    d, V = 1024, 600
    h, w = _normal(3, M, d), _normal(4, V, d)
    hq, hs, _ = m.mosaic_quantize_rows_mxfp4(h)
    wq, ws, _ = m.mosaic_quantize_rows_mxfp4(w)
    far = m.mosaic_quantized_logits_mxfp4(hq, hs + 100, wq, ws - 100, out_dtype=F32)
    near = m.mosaic_quantized_logits_mxfp4(hq, hs, wq, ws, out_dtype=F32)
    assert torch.equal(far, near)
    hs, ws = hs.clone(), ws.clone()
    hs[0, 7], ws[5, 31] = 255, 255
    got = m.mosaic_quantized_logits_mxfp4(hq, hs, wq, ws, out_dtype=F32)
    nan = torch.isnan(got)
    assert bool(nan[0].all()) and bool(nan[:, 5].all())
    nan[0], nan[:, 5] = False, False
    assert not bool(nan.any())
    keep = torch.arange(V, device=DEV) != 5
    assert torch.equal(got[1:][:, keep], near[1:][:, keep])


@pytest.mark.parametrize("M,V,d", [(5, 70, 96), (20, 300, 512), (300, 1000, 512), (70, 257, 1040)])
def test_scales_at_any_address_and_guards(m, M, V, d):
    hq, hs, _ = m.mosaic_quantize_rows_mxfp4(_normal(5, M, d))
    wq, ws, _ = m.mosaic_quantize_rows_mxfp4(_normal(6, V, d))
    want = m.mosaic_quantized_logits_mxfp4(hq, hs, wq, ws)

    def moved(t, by):
        big = torch.full((t.numel() + by,), 255, dtype=torch.uint8, device=DEV)
        big[by:] = t.reshape(-1)
        return big[by:].view(t.shape)
    for by in (1, 2, 3, 7):
        assert torch.equal(m.mosaic_quantized_logits_mxfp4(hq, moved(hs, by), wq, moved(ws, by + 1)), want)
    room = torch.full((M * V + 64,), 3.0, dtype=BF, device=DEV)
    m.mosaic_quantized_logits_mxfp4(hq, hs, wq, ws, out=room[:M * V].view(M, V))
    assert torch.equal(room[:M * V].view(M, V), want) and bool((room[M * V:] == 3).all())


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,V,d", [(33, 33000, 256), (64, 40001, 500), (48, 32769, 1504), (32, 70001, 160), (1, 70000, 544)])
def test_few_rows_of_a_large_vocabulary(m, M, V, d, out):
    test_logits(m, M, V, d, out)
