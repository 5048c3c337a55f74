"""The INT8 head: products of 8-bit codes, against the plain 64-bit form."""
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


SHAPES = [  # (M, V, d): every form at and around its limits
    (1, 1, 1), (1, 1, 16), (3, 5, 7), (64, 64, 64), (65, 63, 65), (77, 1021, 1040), (2, 300, 128), (20, 1000, 128),
    (33, 515, 256), (64, 1030, 384), (65, 1030, 384), (64, 2051, 1024), (255, 257, 128), (256, 256, 256),
    (257, 511, 384), (300, 777, 640), (513, 700, 1024), (700, 513, 4096), (130, 260, 2000), (5, 4099, 3584),
]


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("M,V,d", SHAPES)
def test_int8_logits(m, M, V, d, out_dtype):
    hq, hs = _codes(M + d, M, d)
    wq, ws = _codes(V + d + 1, V, d)
    out = torch.full((M + 1, V), 7.0, dtype=out_dtype, device=DEV)   # the row behind stays as it was
    got = m.mosaic_quantized_logits(hq, hs, wq, ws, out=out)
    plain64.check_int8_logits(got[:M], hq, hs, wq, ws, "logits")
    assert bool((out[M] == 7).all())


@pytest.mark.parametrize("M", [1, 16, 20, 32, 33, 64, 65, 200])
@pytest.mark.parametrize("V,d", [(9000, 128), (5000, 512), (33333, 256), (152064, 128)])
def test_int8_few_rows(m, M, V, d):
    hq, hs = _codes(M, M, d)
    wq, ws = _codes(V, V, d)
    for out_dtype in (BF, F32):
        got = m.mosaic_quantized_logits(hq, hs, wq, ws, out_dtype=out_dtype)
        plain64.check_int8_logits(got, hq, hs, wq, ws, "logits")


@pytest.mark.parametrize("M,V,d", [
    (100, 20000, 256), (128, 16500, 144),                        # 64 x 64 tiles
    (100, 30000, 128), (128, 25000, 384), (65, 80001, 400),      # one row tile of 128 rows, the last with several per CU
    (300, 11000, 128), (300, 11000, 384), (300, 11000, 640),     # 128 x 256 tiles: 1, 3 and 5 K tiles
    (300, 11001, 16), (300, 11001, 272), (300, 11003, 1040),     # ... that the depth does not fill
    (600, 30000, 128), (600, 30000, 256), (600, 30000, 400),     # ... several tiles per workgroup
    (8300, 400, 128), (8300, 400, 640),                          # ... row tiles past a full super-group
    (200, 33000, 128), (200, 33000, 384), (250, 70001, 512),     # one row tile of 256 rows
    (300, 25600, 128), (300, 25600, 384), (300, 25600, 640),     # 256 x 256 tiles: 1, 3 and 5 K tiles
    (300, 25601, 16), (300, 25601, 272), (300, 25603, 1040),     # ... that the depth does not fill
    (1100, 25600, 128), (1100, 25600, 400),                      # ... several tiles per workgroup
    (16484, 600, 128), (16484, 600, 304),                        # ... row tiles past a full super-group
    (40, 700, 8192), (40, 700, 8191), (5, 33, 5008), (250, 1000, 640),   # 32 x 32 tiles
    (20, 9000, 512), (200, 2000, 1024), (250, 3001, 515), (250, 3001, 2064),   # few tiles of 32 x 64 and 64 x 64
    (20, 40001, 259), (32, 33000, 1), (17, 9001, 4099),          # unaligned rows: tiles of 32 rows
    (50, 40001, 259), (64, 33000, 15), (64, 33003, 513),         # ... 64 x 128 tiles
    (300, 7003, 1031), (65, 20000, 17),                          # ... 64 x 64 tiles
    (500, 20000, 515), (130, 33000, 15), (130, 33001, 17), (1300, 2500, 129), (1300, 2501, 127),   # ... 128 x 128 tiles
])
def test_int8_large_tiles(m, M, V, d):
    hq, hs = _codes(M, M, d)
    wq, ws = _codes(V, V, d)
    rows = torch.tensor(sorted({0, 1, 63 % M, 64 % M, 255 % M, 256 % M, M // 2, max(M - 65, 0), M - 2, M - 1}), device=DEV)
    for out_dtype in (BF, F32):
        out = torch.full((M + 1, V), 7.0, dtype=out_dtype, device=DEV)
        got = m.mosaic_quantized_logits(hq, hs, wq, ws, out=out)
        plain64.check_int8_logits(got[rows], hq[rows], hs[rows], wq, ws, "logits")
        assert bool((out[M] == 7).all())
        # every row, against the library's own other form: the same bits
        for r in range(0, M, max(32, M // 8 // 32 * 32)):
            part = m.mosaic_quantized_logits(hq[r:r + 32], hs[r:r + 32], wq, ws, out_dtype=out_dtype)
            assert torch.equal(part, got[r:r + 32][:part.shape[0]])


def test_int8_largest_sums(m):
    # every code -128 at the greatest depth: sums of 131071 * 2^14, next to int32's end
    for d in (131071, 130944):
        hq = torch.full((3, d), -128, dtype=torch.int8, device=DEV)
        wq = torch.full((70, d), -128, dtype=torch.int8, device=DEV)
        one = torch.ones(70, device=DEV)
        got = m.mosaic_quantized_logits(hq, one[:3], wq, one, out_dtype=F32)
        assert bool((got.double() == float(torch.tensor(d * 16384.0, dtype=F32))).all())
    with pytest.raises(m.MosaicError) as e:
        z = torch.zeros((1, 131072), dtype=torch.int8, device=DEV)
        m.mosaic_quantized_logits(z, one[:1], z, one[:1])
    assert e.value.status == m.MOSAIC_ERR_UNSUPPORTED


@pytest.mark.parametrize("M,V,d", [(20, 1000, 256), (40, 3000, 128), (300, 600, 512), (70, 300, 100), (300, 11000, 256), (90, 17000, 128),
                                   (300, 25600, 256), (120, 25600, 256), (200, 33000, 128), (500, 20000, 131),
                                   (50, 33000, 33), (40, 700, 1024), (300, 2000, 1024), (300, 2000, 515)])
def test_int8_device_count(m, M, V, d):
    hq, hs = _codes(1, M, d)
    wq, ws = _codes(2, V, d)
    for out_dtype in (BF, F32):
        want = m.mosaic_quantized_logits(hq, hs, wq, ws, out_dtype=out_dtype)
        for cnt in (-1, 0, 1, 17, M - 1, M, M + 50):
            n = max(0, min(cnt, M))
            out = torch.full((M, V), 5.0, dtype=out_dtype, device=DEV)
            count = torch.tensor([cnt], dtype=torch.int32, device=DEV)
            m.mosaic_quantized_logits(hq, hs, wq, ws, count=count, out=out)
            assert torch.equal(out[:n], want[:n]) and bool((out[n:] == 5).all()), cnt


@pytest.mark.parametrize("M,V,d,off", [(30, 500, 128, 1), (30, 500, 128, 8), (300, 700, 256, 5), (9, 100, 33, 3), (300, 20000, 144, 3), (50, 33000, 128, 1)])
def test_int8_unaligned_codes(m, M, V, d, off):
    hq, hs = _codes(1, M, d)
    wq, ws = _codes(2, V, d)
    want = m.mosaic_quantized_logits(hq, hs, wq, ws, out_dtype=F32)

    def moved(t):   # the same values `off` elements into an allocation
        buf = torch.empty(t.numel() + off, dtype=t.dtype, device=DEV)
        buf[off:] = t.reshape(-1)
        return buf[off:].view(t.shape)

    assert torch.equal(m.mosaic_quantized_logits(moved(hq), moved(hs), moved(wq), moved(ws), out_dtype=F32), want)


def test_int8_zero_scales_and_nan_rows(m):
    hq, hs = _codes(1, 90, 256)
    wq, ws = _codes(2, 300, 256)
    hs[3], hs[5] = 0.0, float("nan")
    ws[7] = 0.0
    got = m.mosaic_quantized_logits(hq, hs, wq, ws)
    assert bool((got[3] == 0).all()) and bool(torch.isnan(got[5]).all()) and bool((got[6, 7] == 0))


@pytest.mark.parametrize("in_dtype", [BF, F32])
@pytest.mark.parametrize("M,V,d,chunk", [(20, 3000, 256, 0), (150, 700, 384, 64), (300, 500, 1000, 128), (1, 9, 5, 0)])
def test_masked_logits_int8(m, M, V, d, chunk, in_dtype):
    g = torch.Generator().manual_seed(M)
    H = torch.randn(2 * M, d, generator=g).to(in_dtype).to(DEV)
    W = (0.02 * torch.randn(V, d, generator=g)).to(in_dtype).to(DEV)
    idx = torch.randint(0, 2 * M, (M,), generator=g, dtype=torch.int32).to(DEV)
    wq, ws = m.mosaic_quantize_rows_int8(W)
    hq, hs = plain64.quantize_int8(H[idx.long()])
    for out_dtype in (BF, F32):
        got = m.mosaic_masked_logits_int8(H, idx, wq, ws, chunk_rows=chunk, out_dtype=out_dtype)
        plain64.check_int8_logits(got, hq, hs, wq, ws, "masked logits")
        whole = m.mosaic_masked_logits_int8(H, idx, wq, ws, out_dtype=out_dtype)
        assert torch.equal(got, whole)


def test_masked_logits_int8_checks_idx_when_asked(m, lib_env):
    H = torch.randn(10, 64, device=DEV)
    wq, ws = m.mosaic_quantize_rows_int8(torch.randn(50, 64, device=DEV))
    idx = torch.tensor([1, 10, 3], dtype=torch.int32, device=DEV)
    got = m.mosaic_masked_logits_int8(H, idx, wq, ws)
    assert bool(torch.isnan(got[1]).all()) and bool(torch.isfinite(got[[0, 2]]).all())
    lib_env("MOSAIC_CHECK_IDX", "1")
    with pytest.raises(m.MosaicError) as e:
        m.mosaic_masked_logits_int8(H, idx, wq, ws)
    assert e.value.status == m.MOSAIC_ERR_INVALID_ARG


@pytest.mark.parametrize("M", [20, 300])
def test_e4m3_codes_in_hand_match_the_fp8_head(m, M):
    H = torch.randn(M, 256, device=DEV).to(BF)
    W = (0.02 * torch.randn(1000, 256, device=DEV)).to(BF)
    wq, ws = m.mosaic_quantize_rows_fp8(W)
    hq, hs = m.mosaic_quantize_rows_fp8(H)
    idx = torch.arange(M, dtype=torch.int32, device=DEV)
    assert torch.equal(m.mosaic_quantized_logits(hq, hs, wq, ws), m.mosaic_masked_logits_fp8(H, idx, wq, ws))
