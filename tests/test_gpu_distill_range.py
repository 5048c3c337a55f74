"""The distillation loss at the ends of its documented range: logits of the type's lowest value
under a teacher's mass."""
import math

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
