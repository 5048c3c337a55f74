"""The MXFP4 head where its large tiles run: bit for bit the rows of small calls, and a sample in 64 bits."""
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


def _codes(seed, n, blocks):
    """Any codes, with scales of 2^-9 to 2^9."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randint(0, 256, (n, 16 * blocks), generator=g, device=DEV, dtype=torch.uint8),
            torch.randint(118, 137, (n, blocks), generator=g, device=DEV, dtype=torch.uint8))


def _same(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def _by_slices(m, hq, hs, wq, ws, out):
    """32 rows a call, which small tiles take."""
    to = torch.empty(hq.shape[0], wq.shape[0], dtype=out, device=DEV)
    for i in range(0, hq.shape[0], 32):
        m.mosaic_quantized_logits_mxfp4(hq[i:i + 32], hs[i:i + 32], wq, ws, out=to[i:i + 32])
    return to


# On 256 CUs: tiles of 128 rows (one row tile, several, and several turns of a workgroup's list with full groups of
# 64 row tiles) and of 256 rows (the same), with the scales of four K tiles together (d a multiple of 512) or
# tile by tile, five K tiles and more, vocabularies with a ragged end, of whole stores and of whole lines.
SHAPES = [
    (128, 70001, 4608), (128, 66048, 1920), (120, 33000, 1152),
    (300, 33001, 4096), (384, 33001, 1920), (300, 33000, 1152),
    (43576, 700, 512), (43576, 704, 640),
    (256, 66048, 4096), (250, 66001, 1152),
    (1229, 13001, 4608), (700, 12001, 1920), (2500, 9000, 1152), (2500, 9001, 4096), (1000, 33024, 1536),
    (16700, 700, 1024), (16700, 4353, 1920),
]


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,V,d", SHAPES)
def test_large_tiles(m, M, V, d, out):
    B = d // 32
    (hq, hs), (wq, ws) = _codes(M + d, M, B), _codes(V + d, V, B)
    got = m.mosaic_quantized_logits_mxfp4(hq, hs, wq, ws, out_dtype=out)
    want = _by_slices(m, hq, hs, wq, ws, out)
    assert torch.equal(got, want)
    g = torch.Generator().manual_seed(M)
    r = torch.cat([torch.randint(0, M, (30,), generator=g), torch.tensor([0, M - 1])]).to(DEV)
    c = torch.cat([torch.randint(0, V, (200,), generator=g), torch.tensor([0, V - 1])]).to(DEV)
    head64.check_mxfp4_logits(got[r][:, c], hq[r], hs[r], wq[c], ws[c], d, f"{M} x {V} x {d}")
    # a count of rows on the device; what lies behind it is left alone
    for n in (0, 1, M // 2 + 3, M - 1):
        to = torch.full_like(got, 3)
        m.mosaic_quantized_logits_mxfp4(hq, hs, wq, ws, count=torch.tensor([n], dtype=torch.int32, device=DEV), out=to)
        assert torch.equal(to[:n], got[:n]) and bool((to[n:] == 3).all())


@pytest.mark.parametrize("M,V,d", [(300, 33001, 1024), (2500, 9001, 4096), (128, 70001, 512), (700, 12001, 1920)])
def test_scales_at_other_addresses_and_guards(m, M, V, d):
    # whole words that are no multiple of 16 bytes, and bytes at any address; outputs that start at any 16 bytes
    B = d // 32
    (hq, hs), (wq, ws) = _codes(1, M, B), _codes(2, V, B)
    want = m.mosaic_quantized_logits_mxfp4(hq, hs, wq, ws)

    def moved(t, by):
        big = torch.full((t.numel() + by,), 255, dtype=torch.uint8, device=DEV)
        big[by:] = t.reshape(-1)
        return big[by:].view(t.shape)
    for a, b in ((4, 0), (0, 8), (12, 4), (1, 6)):
        assert torch.equal(m.mosaic_quantized_logits_mxfp4(hq, moved(hs, a), wq, moved(ws, b)), want), (a, b)
    room = torch.full((8 + M * V + 64,), 3.0, dtype=BF, device=DEV)
    m.mosaic_quantized_logits_mxfp4(hq, hs, wq, ws, out=room[8:8 + M * V].view(M, V))
    assert torch.equal(room[8:8 + M * V].view(M, V), want)
    assert bool((room[:8] == 3).all()) and bool((room[8 + M * V:] == 3).all())


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,V,d", [(300, 33001, 4096), (2500, 9001, 4096), (700, 12001, 1920)])
def test_a_nan_scale_takes_its_row_or_column_alone(m, M, V, d, out):
    B = d // 32
    (hq, hs), (wq, ws) = _codes(3, M, B), _codes(4, V, B)
    near = m.mosaic_quantized_logits_mxfp4(hq, hs, wq, ws, out_dtype=out)
    rows, cols = [0, 129, M - 1], [5, 257, V - 1]
    for k, (i, j) in enumerate(zip(rows, cols)):
        hs[i, (7, 0, B - 1)[k]], ws[j, (B - 1, 31, 0)[k]] = 255, 255
    got = m.mosaic_quantized_logits_mxfp4(hq, hs, wq, ws, out_dtype=out)
    near[rows] = float("nan")
    near[:, cols] = float("nan")
    assert _same(got, near)


def test_masked_rows_in_chunks_of_large_tiles(m):
    L, M, V, d = 3000, 2500, 9001, 1920
    H = torch.randn(L, d, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV).to(BF)
    wq, ws = _codes(6, V, d // 32)
    idx = torch.randint(0, L, (M,), generator=torch.Generator().manual_seed(7)).to(torch.int32).to(DEV)
    hq, hs, _ = m.mosaic_quantize_rows_mxfp4(H, row_idx=idx)
    want = _by_slices(m, hq, hs, wq, ws, BF)
    for C in (0, 2048, 1000, 700):   # (chunks that start off a 16-byte boundary of out)
        assert torch.equal(m.mosaic_masked_logits_mxfp4(H, idx, wq, ws, chunk_rows=C), want), C
