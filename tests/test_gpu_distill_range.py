"""The distillation loss at the ends of its documented range: logits of the type's lowest value
under a teacher's mass, sums over very long rows."""
import math

import pytest
import torch

import device64
import plain64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def m():
    from mask_only_logits_amd import mosaic
    return mosaic


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,V", [(5, 100), (5, 5003), (130, 20000), (5, 152064), (130, 70000), (130, 160001)])
@pytest.mark.parametrize("T", [0.05, 0.5, 0.7, 1.0, 1.9])
def test_loss_of_lowest_logits_under_a_teacher(m, M, V, dtype, T):
    # (z - m) / T passes fp32's range, T^2 times it does not
    low = torch.finfo(dtype).min
    g = torch.Generator().manual_seed(V)
    z = torch.randn(M, V, generator=g).to(dtype)
    t = torch.rand(M, 4, generator=g)
    ids = torch.arange(4, dtype=torch.int32).repeat(M, 1)
    z[:, 1] = low                                    # about a quarter of the mass on it
    z[0, 0:3] = low
    z[1, :] = low                                    # equal logits: nothing special
    z[2, 2] = -math.inf                              # infinite all the same
    t[3, 1] = -math.inf                              # no mass on it: finite and small
    ids[4, 1] = V
    want = plain64.distill(z, t, ids, T)["loss"]
    for loss in (m.mosaic_distill_topk(z.to(DEV), t.to(DEV), ids.to(DEV), temperature=T)[0],
                 m.mosaic_distill_topk(z.to(DEV), t.to(DEV), ids.to(DEV), temperature=T, with_grad=True)[0]):
        got = loss.cpu().double()
        assert math.isinf(float(got[2])) and math.isinf(float(want[2]))
        keep = torch.arange(M) != 2
        keep &= want < 3.4e38                        # what fp32 can hold (T = 1.9, three quarters of the mass)
        # p: 2^6 half steps (arguments of 20 at most, 4 each, for T = 0.05; else fewer); 2^6 for the rest
        size = (2.0 ** 6 + 4 / T * 2) * plain64.U32 * want.abs() + T * T * 2.0 ** -12
        assert ((got - want).abs() <= size)[keep].all(), (got[:5], want[:5])


# rows whose terms are equal, so that every addition may round the same way; each thread meets the
# maximum in its first chunk
@pytest.mark.parametrize("dtype,M,V", [(F32, 1, 1 << 30), (F32, 130, 1 << 24), (F32, 800, 1 << 22), (BF, 1, 1 << 30)])
def test_sums_of_very_long_rows(m, dtype, M, V):
    level = [2.885, 4.26, 4.6975, 3.885, 0.1975] if M == 1 else [(i % 128 + 1) / 16 + 0.01 for i in range(M)]
    parts = 64 if M == 1 else 1                      # what the call splits a row into
    top = 256 * 8 if M == 1 else 1024 * 8
    for first in range(0, len(level), M):
        x = -torch.tensor(level[first:first + M], device=DEV).to(dtype)
        z = x[:, None].expand(M, V).contiguous()
        z.view(M, parts, V // parts)[:, :, :top] = 0.0
        ids = torch.full((M, 1), V - 1, dtype=torch.int32, device=DEV)
        loss, stats, _ = m.mosaic_distill_topk(z, torch.zeros(M, 1, device=DEV), ids)
        n = parts * top
        want = torch.log(n + (V - n) * torch.exp(x.double()))
        # at most 2^9 + 2^8 additions with half a step each (runs of 2^9 chunks, which are joined), the
        # exponential's (3 X + 2), six levels and 64 parts with 5 each, 4 for the logarithm
        tol = (768 + 100 + 3 * x.double().abs() + 4 * want) * plain64.U32
        off = (stats[:, 1].double() - want).abs()
        assert bool((stats[:, 0] == 0).all()) and bool((off <= tol).all()), float((off / plain64.U32).max())
        # one entry with all the mass: the loss is -log q of it, l - x
        assert bool(((loss.double() - (want - x.double())).abs() <= tol + 4 * plain64.U32 * (want - x.double())).all())
        del z


# rows just past one run of a thread's chunks in each form: 16, 8 and 4 waves per row, parts of rows
@pytest.mark.parametrize("dtype,M,V", [(BF, 130, (1 << 22) + 5), (F32, 130, (1 << 21) + 3), (BF, 300, (1 << 21) + 1),
                                       (F32, 300, (1 << 20) + 9), (BF, 800, (1 << 20) + 8), (F32, 800, (1 << 19) + 2),
                                       (F32, 2, (1 << 25) + 64 * 8 + 3), (BF, 2, (1 << 26) + 64 * 8 + 7)])
def test_rows_of_two_runs(m, dtype, M, V):
    g = torch.Generator(device=DEV).manual_seed(V)
    z = torch.empty(M, V, dtype=dtype, device=DEV)
    for i in range(0, M, 16):
        z[i:i + 16] = 2 * torch.randn(min(16, M - i), V, generator=g, device=DEV)
    z[0, V - 1] = 30.0                               # the maximum behind the first run
    z[1, : V - 3] = -math.inf                        # nothing in the first run
    t = 2 * torch.randn(M, 5, generator=g, device=DEV)
    ids = torch.randint(0, V, (M, 5), generator=g, dtype=torch.int32, device=DEV)
    ids[1] = V - 2
    loss, stats, _ = m.mosaic_distill_topk(z, t, ids)
    device64.check_distill(z, t, ids, 1.0, None, loss, stats, None, "loss")
    w = torch.rand(M, generator=g, device=DEV)
    loss, stats, grad = m.mosaic_distill_topk(z, t, ids, with_grad=True, grad_loss=w)
    device64.check_distill(z, t, ids, 1.0, w, loss, stats, grad, "both")
