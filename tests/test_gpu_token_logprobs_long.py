"""Token log-probabilities of rows so long that a workgroup takes its sums in more than one run: 512 chunks of 16 bytes
for each of 256 threads, 2^20 bf16 or 2^19 fp32 logits, in rows too many to be split (more than 512)."""
import math

import pytest
import torch

import head64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
M = 520


@pytest.fixture(scope="module")
def m():
    from mask_only_logits_amd import mosaic
    return mosaic


def _rows(V, dtype):
    """M rows of V logits, the first 13 of them with their largest in chosen places, and a token for each."""
    g = torch.Generator(device=DEV).manual_seed(V)
    z = torch.empty(M, V, dtype=dtype, device=DEV)
    for i in range(0, M, 65):
        z[i:i + 65] = torch.randn(65, V, generator=g, device=DEV).to(dtype)
    n = 8 if dtype == BF else 4                  # logits of a chunk
    run = 512 * 256 * n

    def at(thread, chunk, k=0):                  # the k-th logit of a thread's chunk
        return min((chunk * 256 + thread) * n + k, V - 1)
    last = V // (256 * n) - 1                    # the last round that all threads take
    high = 10 + torch.arange(64, device=DEV) / 4   # 64 values above all others, exact in bf16
    spread = torch.randperm(V - run, generator=torch.Generator().manual_seed(1))[:64].to(DEV)
    z[1, run + spread] = high.to(dtype)          # all in later runs
    one = sorted({at(77, c, c % n) for i in range(32) for c in (3 + 5 * i, 512 + (7 * i) % (last - 511))})
    z[2, torch.tensor(one, device=DEV)] = high[:len(one)].to(dtype)   # all of one thread, in every run
    late = min(last, 520)
    z[3, at(5, 9)], z[3, at(5, late, 1)] = 30.0, 29.0   # a thread's largest first, its second in a later run
    z[4, at(5, 9)], z[4, at(5, late, 1)] = 29.0, 30.0   # and the other way round
    z[5] = (torch.arange(V, device=DEV) / V * 40).to(dtype)            # ascending
    z[6, V - 1] = 50.0                           # the row's last logit
    z[7, run] = 50.0                             # the first of the second run
    z[8, run + 1] = math.nan
    z[9, run + 2] = math.inf
    z[10] = -math.inf
    z[10, run - 1], z[10, run], z[10, V - 1] = 1.0, 1.0, 0.5
    z[11] = -math.inf
    z[12] = 0.0                                  # all equal: the lowest entries
    t = torch.randint(0, V, (M,), generator=g, device=DEV).to(torch.int32)
    t[1], t[6], t[10] = int(run + spread[0]), V - 1, run
    return z, t, g


@pytest.mark.parametrize("dtype,V", [(F32, (1 << 19) + 5003), (F32, (1 << 20) + 2001), (BF, (1 << 20) + 10007),
                                     (BF, (1 << 21) + 4001)])
def test_rows_of_several_runs(m, dtype, V):
    z, t, g = _rows(V, dtype)
    rows = torch.cat([torch.arange(15, device=DEV), torch.tensor([300, M - 1], device=DEV)])
    zs, ts = z[rows], t[rows]
    for n in (0, 2, 20, 64):
        lp, H, ids, top, st = m.mosaic_token_logprobs(z, t, top_n=n, with_entropy=True)
        cut = None if n == 0 else ids[rows], None if n == 0 else top[rows]
        head64.check_logprobs(zs, ts, 1.0, lp[rows], H[rows], *cut, st[rows], f"{V}, {n}")
        lp2, _, ids2, top2, st2 = m.mosaic_token_logprobs(z, t, top_n=n)
        bad = torch.isnan(lp)
        assert torch.equal(lp2[~bad], lp[~bad]) and torch.equal(torch.isnan(lp2), bad)
        if n:
            assert torch.equal(ids, ids2) and torch.equal(torch.nan_to_num(top, 7.0), torch.nan_to_num(top2, 7.0))
    gl, gh = torch.randn(len(rows), generator=g, device=DEV), torch.randn(len(rows), generator=g, device=DEV)
    grad = m.mosaic_token_logprobs_grad(zs, ts, st[rows], gl, entropy=H[rows], grad_entropy=gh)
    head64.check_logprobs_grad(zs, ts, 1.0, gl, gh, grad, f"{V}")
