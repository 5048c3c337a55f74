"""The distillation loss in 64 bits on the GPU, every row of it, with tolerances that go by
element.

U is half a step of fp32, 2^-24.  For one row, with X_v = (m - z_v) / T >= 0, E = sum_v q_v X_v,
x_j = (max t - t_j) / T and e = sum_j p_j x_j, the library's roundings add up to:

* an exponential's argument z c - k in powers of two: c carries two roundings, the fused
  multiply-add one, so the exponential is off by 3 U X of its value, and by two half steps of its
  own: (3 X + 2) U;
* a maximum that a stream of logits raises: the sum so far is multiplied by an exponential of
  the difference (a subtraction, a product with c: 4 U of the difference, which add up to 4 X for
  a term over all the times), and takes two corrections and three products, 9 U a time; at
  most 16 times in these tests' random rows: 4 X + 144;
* additions: three levels in a chunk, one for each chunk of a thread, six levels in a wave and 16
  waves or 64 parts joined, each with a factor that is right to 5 U: at most 100 + chunks;
* so the sum of exponentials is off by ds = (7 E + 250 + chunks) U of its value, and the log-sum l
  by ds and the logarithm's own 4 U l;
* p_j: 4 U x_j + 2 U for its exponential, the same on average and 22 additions for the sum, one
  division: dp_j = (4 x_j + 4 e + 34) U of p_j;
* the gradient T g (q - P): q from the sum (or from exp(l): 6 U l more) and an exponential:
  ds + (3 X + 8 + 6 l) U of q; P dp and the additions of its shares; then one subtraction, a
  product and the rounding to the stored type.
"""
import math

import torch

from plain64 import HALF, TINY, U32


def _rows(z, t, ids, T, g, chunks):
    V = z.shape[1]
    z, t, ids = z.double(), t.double(), ids.long()
    here = (ids >= 0) & (ids < V) & (t != -math.inf)
    any_ = here.any(dim=1)
    tt = torch.where(here, t, torch.full_like(t, -math.inf)) / T
    zero = torch.zeros_like(tt)
    p = torch.where(any_[:, None], torch.softmax(tt, dim=1), zero) if t.shape[1] else tt
    p = torch.where(here, p, zero)
    x = torch.where(p > 0, (tt.amax(dim=1, keepdim=True) - tt).clamp(max=200.0), zero) if t.shape[1] else tt
    e = (p * x).sum(dim=1, keepdim=True)
    dp = (4 * x + 4 * e + 34) * U32
    m = z.amax(dim=1, keepdim=True)
    logq = (z - m) / T
    l = torch.logsumexp(logq, dim=1, keepdim=True)
    X = (-logq).clamp(max=200.0)
    logq = logq - l
    q = torch.exp(logq)
    E = torch.nan_to_num((q * X).sum(dim=1, keepdim=True))
    ds = (7 * E + 250 + chunks) * U32
    dl = ds + 4 * U32 * l.abs()
    idc = ids.clamp(0, V - 1)
    lq = torch.gather(logq, 1, idc)
    cross = torch.where(p > 0, -p * lq, torch.where(p == 0, zero, p))
    lp = torch.where(p > 0, torch.log(torch.where(p > 0, p, torch.ones_like(p))), zero)
    loss = torch.where(any_, T * T * (p * lp + cross).sum(dim=1), torch.zeros_like(l[:, 0]))
    size = p * lp.abs() + cross.abs()
    tol_loss = T * T * ((p * dp * (lp.abs() + 1) + cross.abs() * dp).sum(dim=1) + dl[:, 0] + 40 * U32 * size.sum(dim=1)
                        + 8 * U32 * l[:, 0].abs()) + TINY
    P = torch.zeros_like(z).scatter_add_(1, idc, p)
    dP = torch.zeros_like(z).scatter_add_(1, idc, p * (dp + (2 + t.shape[1]) * U32))
    tg = T * g.double()[:, None]
    grad = torch.where(any_[:, None], tg * (q - P), torch.zeros_like(z))
    tol_grad = tg.abs() * (torch.nan_to_num(q) * (ds + (3 * X + 10 + 6 * l.abs()) * U32) + dP + TINY) + TINY
    return dict(loss=loss, tol_loss=tol_loss, m=m[:, 0], l=l[:, 0], tol_l=dl[:, 0], grad=grad, tol_grad=tol_grad)


def _compare(got, want, tol, what, first):
    got = got.double()
    want = torch.where(want > torch.finfo(torch.float32).max, math.inf, want)   # past fp32's range
    tol = torch.nan_to_num(tol, 0.0, 0.0)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN from row {first} on"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities from row {first} on"
    bad = ((got - want).abs() > tol) & ~nan & ~inf
    if bool(bad.any()):
        at = bad.nonzero()[0].tolist()
        i = tuple(at)
        raise AssertionError(f"{what}: {int(bad.sum())} off, the first in row {first + at[0]} at {at[1:]}: "
                             f"{float(got[i])} for {float(want[i])}, tolerance {float(tol[i])}")


def check_distill(z, t, ids, T, g=None, loss=None, stats=None, grad=None, what=""):
    """Every row of the given outputs against the definition in 64 bits."""
    M, V = z.shape
    g = torch.ones(M, device=z.device) if g is None else g
    n = 16 // z.element_size()
    chunks = V / (n * (64 if V <= 16384 else 256))   # a thread's chunks, in the form with the fewest threads
    step = max(1, (1 << 25) // V)
    for i in range(0, M, step):
        rows = slice(i, min(M, i + step))
        ref = _rows(z[rows], t[rows], ids[rows], T, g[rows], chunks)
        if loss is not None:
            _compare(loss[rows], ref["loss"], ref["tol_loss"], what + " loss", i)
        if stats is not None:
            fine = torch.isfinite(ref["l"])
            assert torch.equal(stats[rows, 0].double()[fine], ref["m"][fine]), f"{what}: maximum from row {i} on"
            _compare(stats[rows, 1][fine], ref["l"][fine], ref["tol_l"][fine], what + " log-sum", i)
        if grad is not None:
            _compare(grad[rows], ref["grad"], ref["tol_grad"] + ref["grad"].abs() * HALF[grad.dtype], what + " gradient", i)
