"""Plain 64-bit forms of the norm, the INT8 head and the distillation loss, on the CPU, and
the tolerances that count the library's roundings (a rounding is off by at most half a step,
finfo(t).eps / 2 of the value)."""
import math

import numpy as np
import torch

U32 = 2.0 ** -24                                       # half a step of fp32
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U32}
TINY = 2.0 ** -120                                     # below this fp32 exponentials may be flushed to zero


def norm(x, r, gain, eps, idx=None):
    """(s, y) in fp64."""
    x = x.cpu().double()
    s = x if r is None else x + r.cpu().double()
    if idx is not None:
        s = s[idx.cpu().long()]
    y = s / torch.sqrt((s * s).mean(dim=1, keepdim=True) + eps) * gain.cpu().double()
    return s, y


# fp32 steps between s and y: each thread adds at most 64 squares one after another, then 10
# levels of the reduction (74 roundings of the sum, halved by the root), and 8 more roundings
# for the mean, the root, the division and the two products: under 64 half steps.
NORM_REL = 64 * U32


def check_norm(got, want, what):
    tol = want.abs() * (HALF[got.dtype] + NORM_REL) + TINY
    bad = (got.cpu().double() - want).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} values off"


def check_codes(q, scale, y, int8, what, rel=NORM_REL):
    """Codes and scales against the unrounded values y [rows, d] they stand for."""
    top = 127.0 if int8 else 448.0
    amax = y.abs().amax(dim=1)
    sc = scale.cpu().double()
    assert ((sc - amax / top).abs() <= (rel + U32) * amax / top + TINY).all(), f"{what}: scale"
    unit = torch.where(amax[:, None] > 0, y / (amax[:, None] / top), torch.zeros_like(y))
    if int8:
        val = q.cpu().double()
        half = torch.full_like(unit, 0.5)
    else:
        val = q.cpu().view(torch.float8_e4m3fn).double()
        half = torch.clamp(unit.abs() * 2.0 ** -4, min=2.0 ** -10)   # half of the smallest step: 2^-9 / 2
    # the unit value carries y's and amax's errors, and two more roundings
    tol = half + unit.abs() * (2 * rel + 3 * U32)
    bad = (val - unit).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} codes off by {float(((val - unit).abs() - half).max())}"


def quantize_int8(x):
    """Codes and scales as documented, each fp32 operation rounded on its own (exact)."""
    x = x.cpu().float().numpy()
    amax = np.abs(x).max(axis=1) if x.shape[1] else np.zeros(x.shape[0], np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        inv = np.where(amax > 0, np.float32(127.0) / amax, np.float32(0.0)).astype(np.float32)
        q = np.rint((x * inv[:, None]).astype(np.float32)).astype(np.int8)
    return torch.from_numpy(q), torch.from_numpy((amax / np.float32(127.0)).astype(np.float32))


def int8_logits(hq, hs, wq, ws):
    acc = hq.cpu().double() @ wq.cpu().double().t()    # exact: |acc| < 2^31
    return acc * hs.cpu().double()[:, None] * ws.cpu().double()


def check_int8_logits(got, hq, hs, wq, ws, what):
    want = int8_logits(hq, hs, wq, ws)
    # the sum's conversion and two products: three roundings
    tol = want.abs() * (HALF[got.dtype] + 4 * U32) + TINY
    bad = (got.cpu().double() - want).abs() > tol
    assert got.shape == want.shape and not bad.any(), f"{what}: {int(bad.sum())} logits off"


def teacher(t, ids, V, T):
    """p [M, K] of the present entries (0 elsewhere), and which rows have any."""
    t, ids = t.cpu().double(), ids.cpu().long()
    here = (ids >= 0) & (ids < V) & (t != -math.inf)
    any_ = here.any(dim=1)
    x = torch.where(here, t / T, torch.full_like(t, -math.inf))
    p = torch.where(any_[:, None], torch.softmax(x, dim=1), torch.zeros_like(t)) if t.shape[1] else t
    return torch.where(here, p, torch.zeros_like(p)), any_


def distill(z, t, ids, T, g=None):
    """Dict of fp64 loss, m, l, grad (per unit of grad_loss times g), p scattered, q."""
    V = z.shape[1]
    z = z.cpu().double()
    p, any_ = teacher(t, ids, V, T)
    m = z.amax(dim=1)
    l = torch.logsumexp((z - m[:, None]) / T, dim=1)
    logq = (z - m[:, None]) / T - l[:, None]
    idc = ids.cpu().long().clamp(0, V - 1)
    zero = torch.zeros_like(p)
    lq = torch.gather(logq, 1, idc)
    cross = torch.where(p > 0, -p * lq, torch.where(p == 0, zero, p))
    ent = torch.where(p > 0, p * torch.log(torch.where(p > 0, p, torch.ones_like(p))), zero)
    loss = T * T * (ent + cross).sum(dim=1)
    loss = torch.where(any_, loss, torch.zeros_like(loss))
    P = torch.zeros_like(z).scatter_add_(1, idc, p)
    q = torch.exp(logq)
    g = torch.ones(z.shape[0], dtype=torch.float64) if g is None else g.cpu().double()
    grad = T * g[:, None] * (q - P)
    grad = torch.where(any_[:, None], grad, torch.zeros_like(grad))
    size = (ent.abs() + cross.abs()).sum(dim=1) + l.abs()
    return dict(loss=loss, m=m, l=l, grad=grad, P=P, q=q, g=g, size=size, T=T)


# l: a thread adds at most 2^9 exponentials one after another here, then 10 levels, and each
# exponential that counts has an argument of magnitude 64 at most (two roundings, times ln 2)
# and an error of its own of two half steps: under 2^10 half steps.
L_ABS = 2.0 ** 10 * U32


def check_distill(ref, loss=None, stats=None, grad=None, what=""):
    T = ref["T"]
    fine = torch.isfinite(ref["l"])
    if stats is not None:
        s = stats.cpu().double()
        assert torch.equal(s[:, 0][fine], ref["m"][fine]), f"{what}: maximum"
        bad = (s[:, 1] - ref["l"]).abs()[fine] > (L_ABS + 2 * U32 * ref["l"].abs())[fine]
        assert not bad.any(), f"{what}: log-sum"
    if loss is not None:
        got, want = loss.cpu().double(), ref["loss"]
        same = torch.isfinite(want)
        assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN losses"
        assert torch.equal(got[~same & ~torch.isnan(want)], want[~same & ~torch.isnan(want)]), f"{what}: inf losses"
        # l's error, the teacher's (the same sums over K <= 1024 entries), and 2^6 roundings of the terms
        tol = T * T * (4 * L_ABS + 64 * U32 * ref["size"])
        bad = (got - want).abs()[same] > tol[same]
        assert not bad.any(), f"{what}: loss {got[same][bad][:4]} for {want[same][bad][:4]}"
    if grad is not None:
        got, want = grad.cpu().double(), ref["grad"]
        assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN gradients"
        # q and the sum of p each carry l's error and their exponent's (64 at most where q counts:
        # below exp(-64) the value itself is under 2^-92); eight roundings more
        tol = (want.abs() * HALF[grad.dtype] +
               T * ref["g"].abs()[:, None] * (ref["q"] + ref["P"]) * (4 * L_ABS) + TINY +
               T * ref["g"].abs()[:, None] * 2.0 ** -90)
        bad = ((got - want).abs() > tol) & ~torch.isnan(want)
        assert not bad.any(), f"{what}: {int(bad.sum())} gradients off"
