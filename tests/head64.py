"""Plain 64-bit forms of the layer norm, the MXFP4 codes and head and the token
log-probabilities, with tolerances that count the library's roundings (U32 is half a step of
fp32; a rounding to the stored type is off by HALF of the value)."""
import math

import torch

from plain64 import HALF, TINY, U32


def _check(got, want, tol, what):
    got = got.to(want.device).double()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)} for {tuple(want.shape)}"
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN at other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities"
    bad = ((got - want).abs() > torch.nan_to_num(tol, 0.0)) & ~nan & ~inf
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} off, the first at {i}: {float(got[i])} for {float(want[i])}, "
                             f"tolerance {float(tol[i])}")


# ---------------------------------------------------------------------- layer norm ---

def check_layernorm(x, r, gain, bias, eps, idx=None, sum_out=None, out=None, stats=None, what=""):
    """x + r is one rounding of s where there is an r; mean and deviation carry the mean of those.
    fp64's own share: sums of d terms against a variance that is at least 1 / (d + 1) of
    them, additions d / 64 deep at most, with 16 more to join threads."""
    eps = float(torch.tensor(eps, dtype=torch.float32))   # as the library takes it
    x = x.double()
    s = x if r is None else x + r.double()
    e = torch.zeros_like(s) if r is None else U32 * s.abs()
    if idx is not None:
        s, e = s[idx.long()], e[idx.long()]
    d = s.shape[1]
    mu = s.mean(1, keepdim=True)
    u = s - mu
    var = (u * u).mean(1, keepdim=True)
    rho = 1 / torch.sqrt(var + eps)
    xh = u * rho
    e = e + e.mean(1, keepdim=True)
    deep = (d + 1) * (d / 64 + 16) * 2.0 ** -53
    e_rho = rho ** 2 * (u.abs() * e).mean(1, keepdim=True) + deep       # relative
    g = torch.ones(d, dtype=torch.float64, device=s.device) if gain is None else gain.double()
    b = torch.zeros(d, dtype=torch.float64, device=s.device) if bias is None else bias.double()
    y = xh * g + b
    dxh = rho * e + xh.abs() * (e_rho + 2 * U32) + rho * deep * u.abs().mean(1, keepdim=True)
    if sum_out is not None:
        _check(sum_out, s, s.abs() * (HALF[sum_out.dtype] + U32) + TINY, what + " sum")
    if out is not None:
        _check(out, y, dxh * g.abs() + y.abs() * (HALF[out.dtype] + U32) + 2 * U32 * (xh * g).abs() + TINY, what + " out")
    if stats is not None:
        _check(stats[:, :1], mu, e.mean(1, keepdim=True) + deep * s.abs().amax(1, keepdim=True) + TINY, what + " mean")
        _check(stats[:, 1:], rho, rho * (e_rho + 2.0 ** -50), what + " rstd")


def check_layernorm_grad(dy, s, stats, gain, idx=None, dsum=None, dx=None, dgain=None, dbias=None, what=""):
    """The means over a row: a thread adds at most 64 terms one after another, then 10 levels;
    the sums over rows: at most 128 rows in fp32, which are then added in fp64."""
    dy, s = dy.double(), s.double()
    if idx is not None:
        s = s[idx.long()]
    d = dy.shape[1]
    mu, rho = stats[:, :1].double(), stats[:, 1:].double()
    g = torch.ones(d, dtype=torch.float64, device=s.device) if gain is None else gain.double()
    xh, a = (s - mu) * rho, dy * g
    c1, c2 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
    want = rho * (a - c1 - xh * c2)
    tol = rho * U32 * (5 * (a.abs() + c1.abs() + (xh * c2).abs()) + 80 * a.abs().mean(1, keepdim=True) +
                       84 * xh.abs() * (a * xh).abs().mean(1, keepdim=True))
    if dsum is not None:
        want = want + dsum.double()
    if dx is not None:
        _check(dx, want, tol + want.abs() * (HALF[dx.dtype] + 2 * U32) + TINY, what + " dx")
    if dgain is not None:
        _check(dgain, (dy * xh).sum(0), 134 * U32 * (dy * xh).abs().sum(0) + TINY, what + " dgain")
    if dbias is not None:
        _check(dbias, dy.sum(0), 130 * U32 * dy.abs().sum(0) + TINY, what + " dbias")


# --------------------------------------------------------------------------- MXFP4 ---

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def mxfp4_codes(x):
    """(packed codes [n, 16 B], scale bytes [n, B]) of rows, exactly."""
    x = x.detach().cpu().double()
    n, d = x.shape
    B = -(-d // 32)
    b = torch.zeros(n, B * 32, dtype=torch.float64)
    b[:, :d] = x
    b = b.view(n, B, 32)
    amax = b.abs().amax(dim=2)
    fine = torch.isfinite(b).all(dim=2)
    e = torch.where(amax > 0, torch.frexp(torch.where(fine, amax, torch.ones_like(amax))).exponent - 3, -127)
    e = e.clamp(-127, 127)
    y = torch.where(fine[:, :, None], b, torch.zeros_like(b)).abs() * torch.exp2(-e.double())[:, :, None]
    dist = (y[..., None] - E2M1).abs()
    near = dist.amin(dim=-1, keepdim=True)
    tie = (dist == near) & (torch.arange(8) % 2 == 0)
    code = torch.where(tie.any(-1), tie.int().argmax(-1), (dist == near).int().argmax(-1))
    sign = torch.where(fine[:, :, None], torch.signbit(b), torch.zeros_like(b, dtype=torch.bool))
    code = (code + 8 * sign.long()).view(n, B * 16, 2)
    q = (code[:, :, 0] + 16 * code[:, :, 1]).to(torch.uint8)
    return q, torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)


def mxfp4_values(q, scale, d):
    """What codes and scales stand for, [n, d] fp64."""
    q, scale = q.cpu(), scale.cpu()
    table = torch.cat([E2M1, -E2M1])
    v = torch.stack([table[(q & 15).long()], table[(q >> 4).long()]], dim=2).view(q.shape[0], scale.shape[1], 32)
    s = torch.exp2(scale.double() - 127)
    s = torch.where(scale == 255, torch.full_like(s, math.nan), s)
    return (v * s[:, :, None]).view(q.shape[0], -1)[:, :d]


def check_mxfp4_logits(got, hq, hs, wq, ws, d, what=""):
    """Products of codes are exact; each of d additions is off by a step (two half steps, should
    the matrix unit cut instead of round) of a sum that stays below that of the magnitudes."""
    h, w = mxfp4_values(hq, hs, d), mxfp4_values(wq, ws, d)
    want = h @ w.t()
    tol = want.abs() * HALF[got.dtype] + 2 * U32 * (d + 8) * (h.abs() @ w.abs().t()) + TINY
    _check(got.cpu(), want, tol, what)


# -------------------------------------------------------------- token log-probabilities ---
#
# With X_v = (m - z_v) / T: the exponential of X_v is off by (3 X + 2) half steps of its value (two
# roundings of c, one of the fused multiply-add, two half steps of its own); a maximum that rises
# costs a term 4 X over all the times and 12 a time, 16 times at most; additions: three levels in a
# chunk, one for each of a thread's chunks, six levels in a wave, 64 parts joined with factors right to
# five: 100 + chunks.  So the sum is off by ds = (7 E + 300 + chunks) U, E = sum p X, and the log-sum by ds
# and its own 4 U l.  The sum of p X carries the same for each of its terms, and a term's X three
# roundings.

def _rows(z, T, chunks):
    z = z.double()
    m = z.amax(1, keepdim=True)
    x = (z - m) / T
    bad = torch.isnan(z).any(1) | (m[:, 0] == math.inf) | (m[:, 0] == -math.inf)
    l = torch.logsumexp(x, 1, keepdim=True)
    l[bad] = math.nan
    logp = x - l
    p = torch.exp(logp)
    X = (-x).clamp(max=200.0)
    px = torch.where(p > 0, p * -x, torch.zeros_like(p))
    E = px.sum(1, keepdim=True)
    ds = (7 * E + 300 + chunks) * U32
    dl = ds + 4 * U32 * l.abs()
    H = l + E
    dH = dl + ds * E + (torch.where(p > 0, p * X * (7 * X + 308 + chunks), torch.zeros_like(p))).sum(1, keepdim=True) * U32
    dH = dH + 4 * U32 * (l.abs() + E)
    H[bad] = math.nan
    return dict(m=m, l=l, logp=logp, p=p, X=X, E=E, ds=ds, dl=dl, H=H, dH=dH, bad=bad, x=x)


def _chunks(z):
    V, n = z.shape[1], 16 // z.element_size()
    return V / (n * 64)


def check_logprobs(z, tokens, T, logprob=None, entropy=None, top_ids=None, top_logprobs=None, stats=None, what=""):
    """Every given output, row by row; the alternatives are exact."""
    M, V = z.shape
    step = max(1, (1 << 25) // V)
    for i in range(0, M, step):
        k = slice(i, min(M, i + step))
        r = _rows(z[k], T, _chunks(z))
        w = f"{what} from row {i} on:"
        if stats is not None:
            fine = ~r["bad"]
            assert torch.equal(stats[k, 0].double()[fine], r["m"][fine, 0]), f"{w} maximum"
            _check(stats[k, 1], r["l"][:, 0], r["dl"][:, 0] + TINY, w + " log-sum")
        if logprob is not None:
            t = tokens[k].long()
            here = (t >= 0) & (t < V)
            at = t.clamp(0, V - 1)[:, None]
            want, x = r["logp"].gather(1, at)[:, 0], r["x"].gather(1, at)[:, 0]
            want = torch.where(r["bad"], torch.full_like(want, math.nan), want)
            want = torch.where(here, want, torch.zeros_like(want))
            want = torch.where(want < -torch.finfo(torch.float32).max, -math.inf, want)   # past fp32's range
            _check(logprob[k], want, r["dl"][:, 0] + 4 * U32 * (x.abs() + want.abs()) + TINY, w + " logprob")
        if entropy is not None:
            _check(entropy[k], r["H"][:, 0], r["dH"][:, 0] + TINY, w + " entropy")
        if top_ids is not None:
            n = top_ids.shape[1]
            zz = torch.where(r["bad"][:, None], torch.full_like(z[k], -math.inf), z[k]).double() + 0.0
            v, ids = torch.sort(zz, dim=1, descending=True, stable=True)
            v, ids = v[:, :n], ids[:, :n]
            if n > V:
                v = torch.nn.functional.pad(v, (0, n - V), value=-math.inf)
                ids = torch.nn.functional.pad(ids, (0, n - V))
            ids = torch.where(v == -math.inf, torch.full_like(ids, -1), ids)
            assert torch.equal(top_ids[k].long(), ids), f"{w} alternatives"
            x = (v - r["m"]) / T
            want = torch.where(r["bad"][:, None], torch.full_like(x, math.nan),
                               torch.where(ids < 0, torch.full_like(x, -math.inf), x - r["l"]))
            want = torch.where(want < -torch.finfo(torch.float32).max, -math.inf, want)
            _check(top_logprobs[k], want, r["dl"] + 4 * U32 * (x.abs() + want.abs()) + TINY, w + " alternatives")


def check_logprobs_grad(z, tokens, T, g, h, grad, what=""):
    """Against the definition; p carries the log-sum's error, its exponent's and exp(l)'s."""
    M, V = z.shape
    step = max(1, (1 << 24) // V)
    for i in range(0, M, step):
        k = slice(i, min(M, i + step))
        r = _rows(z[k], T, _chunks(z))
        p = r["p"]
        gg = torch.zeros(p.shape[0], 1, dtype=torch.float64, device=z.device)
        hh = gg.clone() if h is None else h[k].double()[:, None]
        delta = torch.zeros_like(p)
        if tokens is not None:
            t = tokens[k].long()
            here = (t >= 0) & (t < V)
            gg = torch.where(here, g[k].double(), torch.zeros_like(gg[:, 0]))[:, None]
            delta.scatter_(1, t.clamp(0, V - 1)[:, None], here.double()[:, None])
        A = torch.where(p > 0, r["logp"] + r["H"], torch.zeros_like(p))
        want = (gg * (delta - p) - hh * p * A) / T
        want[r["bad"]] = math.nan
        dp = r["ds"] + 4 * U32 * r["l"].abs() + (3 * r["X"] + 12 + 6 * r["l"].abs()) * U32
        dA = r["dl"] + r["dH"] + 4 * U32 * (r["X"] + r["l"].abs() + r["H"].abs()) + 3 * U32 * r["X"]
        tol = ((gg.abs() + hh.abs() * A.abs()) * p * dp + hh.abs() * p * dA +
               6 * U32 * (gg.abs() * (delta + p) + hh.abs() * p * A.abs())) / T
        _check(grad[k], want, tol + want.abs() * HALF[grad.dtype] + (gg.abs() + hh.abs()) / T * 2.0 ** -100 + TINY,
               f"{what} gradient from row {i} on")
