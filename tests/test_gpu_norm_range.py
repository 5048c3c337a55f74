"""The norm over its whole documented range: any eps, rows too long for the registers with every
option, all combinations of outputs."""
import itertools

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


def _data(seed, n, d, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, d, generator=g).to(dtype)
    r = (torch.randn(n, d, generator=g) * torch.exp(0.5 * torch.randn(d, generator=g))).to(dtype)
    return x.to(DEV), r.to(DEV), (1 + 0.2 * torch.randn(d, generator=g)).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 1000, 4096, 16384, 16385, 20001])
def test_norm_large_eps_beside_overflowing_squares(m, d, dtype):
    # the squares' sum, or the mean plus eps, passes fp32's range while eps still counts
    for size, eps in ((2.0 ** 62, 1e38), (2.0 ** 62, 1e36), (1.7e19, 3e38), (1e19, 3.4e38), (3e38, 3.4e38), (1.0, 3.4e38),
                      (2.0 ** 61, 1e-6), (2.0 ** 60, 1e33), (2.0 ** 60, 3.4e38)):
        x = (torch.randn(3, d, generator=torch.Generator().manual_seed(d)).clamp(-1, 1) * size).to(dtype).to(DEV)
        gain = torch.ones(d, dtype=dtype, device=DEV)
        _, y, q, sc = m.mosaic_add_rmsnorm(x, gain, eps=eps, code=m.MOSAIC_INT8)
        eps32 = float(torch.tensor(eps, dtype=F32))
        want = plain64.norm(x, None, gain, eps32)[1]
        plain64.check_norm(y, want, f"{size} with eps {eps}")
        plain64.check_codes(q, sc, want, True, f"{size} with eps {eps}")


@pytest.mark.parametrize("dtype,d", [(F32, 1 << 20), (F32, (1 << 24) + 3), (BF, (1 << 24) + 3)])
def test_norm_sums_of_very_long_rows(m, dtype, d):
    # equal elements, so that every addition may round the same way
    for v in (0.1, 0.3, 0.7, 1.1, 1.3, 1.7):
        x = torch.full((1, d), v, dtype=dtype, device=DEV)
        gain = torch.ones(d, dtype=dtype, device=DEV)
        _, y, q, sc = m.mosaic_add_rmsnorm(x, gain, code=m.MOSAIC_INT8)
        want = plain64.norm(x[:, :1], None, gain[:1], 1e-6)[1].to(DEV)
        tol = want.abs() * (plain64.HALF[dtype] + plain64.NORM_REL)
        assert bool(((y.double() - want).abs() <= tol).all()), float((y.double() / want - 1).abs().max() / plain64.U32)
        assert bool((q == 127).all())
        assert bool(((sc.double() * 127 / want[0] - 1).abs() <= plain64.NORM_REL).all())


LONG = [16385, 16392, 20001]


@pytest.mark.parametrize("d", LONG)
def test_long_norm_special_rows(m, d):
    x = torch.randn(8, d, device=DEV)
    x[0] = 0
    x[1, d // 2] = float("nan")
    x[2, 3] = float("inf")
    x[3] = torch.finfo(F32).max
    x[4] *= 1e-30
    x[5] = 0
    x[5, d - 1] = -2.0
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


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", LONG)
def test_long_norm_strides_and_in_place(m, d, dtype):
    x, r, gain = _data(d, 5, d + 24, dtype)
    gain = gain[:d].contiguous()
    for off in (0, 8, 3):
        xs, rs = x[:, off:off + d], r[:, off:off + d]
        ws, wy = plain64.norm(xs, rs, gain, 1e-5)
        wide = torch.full((5, d + 40), 7.0, dtype=dtype, device=DEV)
        s, y, q, sc = m.mosaic_add_rmsnorm(xs, gain, eps=1e-5, residual=rs, sum_out=wide[:, 8:8 + d], code=m.MOSAIC_INT8)
        plain64.check_norm(s, ws, "sum")
        plain64.check_norm(y, wy, "out")
        plain64.check_codes(q, sc, wy, True, "codes")
        assert bool((wide[:, :8] == 7).all()) and bool((wide[:, 8 + d:] == 7).all())
        for into in (0, 1):
            xc, rc = x.clone(), r.clone()
            xv, rv = xc[:, off:off + d], rc[:, off:off + d]
            got = m.mosaic_add_rmsnorm(xv, gain, eps=1e-5, residual=rv, sum_out=(xv, rv)[into], code=m.MOSAIC_INT8)
            for a, b in zip(got, (s, y, q, sc)):
                assert torch.equal(a, b)
            for now, before in ((xc, x), (rc, r)):
                assert torch.equal(now[:, :off], before[:, :off]) and torch.equal(now[:, off + d:], before[:, off + d:])
            assert torch.equal((rc, xc)[into], (r, x)[into])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", LONG)
def test_long_norm_gathered_with_a_device_count(m, d, dtype):
    x, r, gain = _data(d, 11, d, dtype)
    idx = torch.tensor([10, 0, 0, -1, 11, 5, 2**31 - 1, 7], dtype=torch.int32, device=DEV)
    ok, bad = [0, 1, 2, 5, 7], [3, 4, 6]
    ref = m.mosaic_add_rmsnorm(x, gain, residual=r, row_idx=idx, store_sum=True, code=m.MOSAIC_E4M3)
    ws, wy = plain64.norm(x, r, gain, 1e-6, idx[ok])
    plain64.check_norm(ref[0][ok], ws, "sum")
    plain64.check_norm(ref[1][ok], wy, "out")
    plain64.check_codes(ref[2][ok], ref[3][ok], wy, False, "codes")
    assert all(bool(torch.isnan(t[bad]).all()) for t in (ref[0], ref[1], ref[3])) and bool((ref[2][bad] == 0).all())
    for cnt in (-5, 0, 1, 3, 8, 99):
        n = max(0, min(cnt, 8))
        outs = [torch.full_like(t, 9) for t in ref]
        count = torch.tensor([cnt], dtype=torch.int32, device=DEV)
        m.mosaic_add_rmsnorm(x, gain, residual=r, row_idx=idx, count=count, sum_out=outs[0], out=outs[1],
                             code=m.MOSAIC_E4M3, q=outs[2], scale=outs[3])
        for got, want in zip(outs, ref):
            assert torch.equal(got[:n].float().nan_to_num(77.0), want[:n].float().nan_to_num(77.0))
            assert bool((got[n:] == 9).all())


# a width of each form: 8, 16 and 32 threads per row, a wave, two to eight waves, and read again
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [40, 100, 150, 300, 700, 1000, 1100, 2000, 2300, 4000, 5000, 8000, 12000, 17000])
def test_norm_every_combination_of_outputs(m, d, dtype):
    x, r, gain = _data(d, 7, d, dtype)
    for residual in (r, None):
        for code in (m.MOSAIC_INT8, m.MOSAIC_E4M3):
            whole = m.mosaic_add_rmsnorm(x, gain, residual=residual, store_sum=True, code=code)
            ws, wy = plain64.norm(x, residual, gain, 1e-6)
            plain64.check_norm(whole[0], ws, "sum")
            plain64.check_norm(whole[1], wy, "out")
            plain64.check_codes(whole[2], whole[3], wy, code == m.MOSAIC_INT8, "codes")
            for want_sum, want_out, want_q in itertools.product((False, True), repeat=3):
                if not (want_sum or want_out or want_q):
                    continue
                got = m.mosaic_add_rmsnorm(x, gain, residual=residual, store_sum=want_sum, store_out=want_out,
                                           code=code if want_q else None)
                asked = (want_sum, want_out, want_q, want_q)
                for a, b, c in zip(got, whole, asked):
                    assert (a is None) if not c else torch.equal(a, b)
