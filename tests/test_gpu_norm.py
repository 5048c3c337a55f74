"""Residual addition with RMS norm and 8-bit codes, against the plain 64-bit form."""
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


def _data(seed, n, d, dtype, gain_dtype=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, d, generator=g).to(dtype)
    r = (torch.randn(n, d, generator=g) * torch.exp(0.5 * torch.randn(d, generator=g))).to(dtype)
    gain = (1 + 0.2 * torch.randn(d, generator=g)).to(gain_dtype or dtype)
    return x.to(DEV), r.to(DEV), gain.to(DEV)


# widths at and around each form's limits, aligned and not
WIDTHS = [1, 2, 7, 8, 63, 64, 65, 504, 512, 513, 520, 1021, 1024, 1032, 2040, 2048, 2049, 2056, 3584, 4096, 4104,
          8192, 8193, 8200, 16384, 16392, 20001, 127, 128, 129, 191, 192, 193, 256, 257, 383, 384, 385, 767, 768, 769,
          1025, 1535, 1536, 1537, 2559, 2560, 2561, 4097, 6143, 6144, 6145]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", WIDTHS)
def test_norm_widths(m, d, dtype):
    x, r, gain = _data(d, 5, d, dtype)
    for code in (m.MOSAIC_INT8, m.MOSAIC_E4M3):
        s, y, q, sc = m.mosaic_add_rmsnorm(x, gain, residual=r, store_sum=True, code=code)
        ws, wy = plain64.norm(x, r, gain, 1e-6)
        plain64.check_norm(s, ws, "sum")
        plain64.check_norm(y, wy, "out")
        plain64.check_codes(q, sc, wy, code == m.MOSAIC_INT8, "codes")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [1, 64, 65, 128, 150, 192, 255, 384, 700])
def test_norm_narrow_rows_share_a_wave(m, d, dtype):
    # each row as if it were alone, whatever its neighbours hold, at counts that end inside a wave
    x, r, gain = _data(d, 1003, d, dtype)
    r[5::7] = float("nan")
    r[6::11] = torch.finfo(dtype).max
    for rows in (1, 2, 9, 33, 1003):
        idx = torch.randperm(1003, generator=torch.Generator().manual_seed(rows))[:rows].to(torch.int32).to(DEV)
        got = m.mosaic_add_rmsnorm(x, gain, residual=r, row_idx=idx, store_sum=True, code=m.MOSAIC_INT8)
        for i in sorted({0, rows // 3, rows // 2, rows - 1}):
            alone = m.mosaic_add_rmsnorm(x, gain, residual=r, row_idx=idx[i:i + 1], store_sum=True, code=m.MOSAIC_INT8)
            for a, b in zip(got, alone):
                assert torch.equal(a[i:i + 1].nan_to_num(7.0), b.nan_to_num(7.0))
        fine = ~torch.isnan(r[idx.long()]).any(1) & (r[idx.long()].abs() < 1e30).all(1)
        ws, wy = plain64.norm(x, r, gain, 1e-6, idx)
        keep = fine.to(wy.device)
        plain64.check_norm(got[1][fine], wy[keep], "out")
        plain64.check_codes(got[2][fine], got[3][fine], wy[keep], True, "codes")


@pytest.mark.parametrize("dtype,gain_dtype", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("rows", [1, 3, 4, 5, 130])
def test_norm_gathered(m, rows, dtype, gain_dtype):
    x, r, gain = _data(rows, 70, 640, dtype, gain_dtype)
    idx = torch.randint(0, 70, (rows,), dtype=torch.int32, device=DEV)   # repeats among them
    s, y, q, sc = m.mosaic_add_rmsnorm(x, gain, residual=r, row_idx=idx, store_sum=True, code=m.MOSAIC_INT8)
    ws, wy = plain64.norm(x, r, gain, 1e-6, idx)
    plain64.check_norm(s, ws, "sum")
    plain64.check_norm(y, wy, "out")
    plain64.check_codes(q, sc, wy, True, "codes")
    s, y, q, sc = m.mosaic_add_rmsnorm(x, gain, row_idx=idx, store_out=False, code=m.MOSAIC_E4M3)
    assert s is None and y is None
    plain64.check_codes(q, sc, plain64.norm(x, None, gain, 1e-6, idx)[1], False, "codes alone")


@pytest.mark.parametrize("d", [256, 4096, 1000, 1023, 9000, 50, 150, 2500, 5000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_strides_and_in_place(m, d, dtype):
    x, r, gain = _data(d, 9, d + 24, dtype)
    gain = gain[:d].contiguous()
    for off in (0, 8, 3):   # rows inside a wider array: aligned, and one that is not
        xs, rs = x[:, off:off + d], r[:, off:off + d]
        wide = torch.full((9, d + 40), 7.0, dtype=dtype, device=DEV)
        ws, wy = plain64.norm(xs, rs, gain, 1e-5)
        s, y, _, _ = m.mosaic_add_rmsnorm(xs, gain, eps=1e-5, residual=rs, sum_out=wide[:, 8:8 + d])
        plain64.check_norm(s, ws, "sum")
        plain64.check_norm(y, wy, "out")
        assert bool((wide[:, :8] == 7).all()) and bool((wide[:, 8 + d:] == 7).all())
        for into in (0, 1):   # the residual stream updated in place, or x itself
            xc, rc = x.clone(), r.clone()
            xv, rv = xc[:, off:off + d], rc[:, off:off + d]
            s, y2, _, _ = m.mosaic_add_rmsnorm(xv, gain, eps=1e-5, residual=rv, sum_out=(xv, rv)[into])
            plain64.check_norm((xv, rv)[into], ws, "sum in place")
            assert torch.equal(y, y2)


@pytest.mark.parametrize("d", [512, 4096, 1001, 10000, 40, 100, 150, 250, 300])
def test_norm_special_rows(m, d):
    x = torch.randn(8, d, device=DEV)
    x[0] = 0
    x[1, d // 2] = float("nan")
    x[2, 3] = float("inf")
    x[3] = torch.finfo(F32).max            # squares past fp32's range
    x[4] *= 1e-30                          # squares below it: eps decides
    x[5] = 0
    x[5, 7] = -2.0
    x[6] *= 1e25
    gain = torch.ones(d, device=DEV)
    ok = [0, 3, 4, 5, 6, 7]
    for code in (m.MOSAIC_INT8, m.MOSAIC_E4M3):
        _, y, q, sc = m.mosaic_add_rmsnorm(x, gain, code=code)
        want = plain64.norm(x, None, gain, 1e-6)[1]
        plain64.check_norm(y[ok], want[ok], "special rows")
        plain64.check_codes(q[ok], sc[ok], want[ok], code == m.MOSAIC_INT8, "special rows")
        assert torch.isnan(y[1]).all() and torch.isnan(sc[1]) and bool((q[1] == 0).all())
        assert torch.isnan(sc[2]) and bool((q[2] == 0).all())
        assert float(sc[0]) == 0 and bool((q[0] == 0).all())


def test_norm_row_id_outside_gives_nan(m):
    x, _, gain = _data(5, 6, 512, BF)
    idx = torch.tensor([0, -1, 5, 6, 2**31 - 1, 3], dtype=torch.int32, device=DEV)
    _, y, q, sc = m.mosaic_add_rmsnorm(x, gain, row_idx=idx, code=m.MOSAIC_INT8)
    ok, bad = [0, 2, 5], [1, 3, 4]
    plain64.check_norm(y[ok], plain64.norm(x, None, gain, 1e-6)[1][[0, 5, 3]], "valid rows")
    assert torch.isnan(y[bad]).all() and torch.isnan(sc[bad]).all() and bool((q[bad] == 0).all())


@pytest.mark.parametrize("d", [320, 2048, 777, 9001])
def test_norm_device_count(m, d):
    x, r, gain = _data(d, 40, d, BF)
    ref = m.mosaic_add_rmsnorm(x, gain, residual=r, store_sum=True, code=m.MOSAIC_INT8)
    for cnt in (-5, 0, 1, 17, 40, 99):
        n = max(0, min(cnt, 40))
        outs = [torch.full_like(t, 9) for t in ref]
        count = torch.tensor([cnt], dtype=torch.int32, device=DEV)
        m.mosaic_add_rmsnorm(x, gain, residual=r, count=count, sum_out=outs[0], out=outs[1], code=m.MOSAIC_INT8,
                             q=outs[2], scale=outs[3])
        for got, want in zip(outs, ref):
            assert torch.equal(got[:n], want[:n]) and bool((got[n:] == 9).all())


def test_norm_past_32_bit_offsets(m):
    # 2^31 and more elements: rows at both ends of the array
    d, n = 4096, (1 << 31) // 4096 + 300
    x = torch.zeros(n, d, dtype=BF, device=DEV)
    rows = torch.tensor([0, n - 1, n - 2, 1 << 18], dtype=torch.int32, device=DEV)
    x[rows.long()] = torch.randn(4, d, device=DEV).to(BF)
    gain = torch.ones(d, dtype=BF, device=DEV)
    _, y, _, _ = m.mosaic_add_rmsnorm(x, gain, row_idx=rows)
    plain64.check_norm(y, plain64.norm(x[rows.long()], None, gain, 1e-6)[1], "far rows")
    _, y, _, _ = m.mosaic_add_rmsnorm(x, gain)
    plain64.check_norm(y[rows.long()], plain64.norm(x[rows.long()], None, gain, 1e-6)[1], "far results")
    assert float(y[12345].abs().max()) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [1, 8, 100, 512, 1024, 4096, 4097, 20000])
def test_quantize_rows_int8_exact(m, d, dtype):
    g = torch.Generator().manual_seed(d)
    x = (torch.randn(11, d, generator=g) * torch.logspace(-20, 20, 11)[:, None]).to(dtype)
    x[3] = 0
    x[4] = x[4] * 1e-38 * 1e20             # near fp32's smallest normal values
    q, sc = m.mosaic_quantize_rows_int8(x.to(DEV))
    wq, wsc = plain64.quantize_int8(x)
    normal = wsc > 1e-36
    assert torch.equal(sc.cpu()[normal], wsc[normal]) and torch.equal(q.cpu()[normal], wq[normal])
    assert float(sc[3]) == 0 and bool((q[3] == 0).all())
    idx = torch.tensor([10, 0, 0, 5, -3, 11], dtype=torch.int32, device=DEV)
    q2, sc2 = m.mosaic_quantize_rows_int8(x.to(DEV), row_idx=idx)
    assert torch.equal(q2[:4], q[[10, 0, 0, 5]]) and torch.equal(sc2[:4], sc[[10, 0, 0, 5]])
    assert torch.isnan(sc2[4:]).all() and bool((q2[4:] == 0).all())


def test_norm_other_stream(m):
    x, r, gain = _data(1, 2000, 4096, BF)
    want = m.mosaic_add_rmsnorm(x, gain, residual=r, store_sum=True, code=m.MOSAIC_INT8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = m.mosaic_add_rmsnorm(x, gain, residual=r, store_sum=True, code=m.MOSAIC_INT8, stream=stream)
        s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
