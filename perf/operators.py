"""Cases of the operators around the masked rows' LM head: what they are measured on.

Three operators, each with its plain form in elementary torch operations (run with
``own`` false) and as calls of this library (``own`` true):

* ``norm``     residual addition and root-mean-square norm of (gathered) rows, with the
               sum, the normed rows and 8-bit codes (E4M3 or INT8, one scale per row) as
               outputs;
* ``int8``     the matrix product of 8-bit integer codes with a scale per row (token) and
               per vocabulary entry (channel); ``from_h``: the codes of the masked rows
               are made from the hidden states within the call;
* ``distill``  the loss against a teacher's top logits over the masked rows' logits, its
               gradient, or both.

Codes are returned as values: E4M3 codes in torch's own type for them, INT8 codes in
bfloat16 (which holds them all); a row's true values are these times its scale.
"""
import math

import torch

own = False

_E4M3_MAX, _INT8_MAX = 448.0, 127.0
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------- cases ---

def listed():
    return [
        # the 20 masked rows left near the end of a denoising of a 4096-token sequence, int8 head next: latency
        dict(name="norm_few_int8", op="norm", rows=20, src=4096, d=3584, dtype="bf16", residual=True, gather=True,
             store_sum=False, store_out=False, code="int8"),
        # one denoising step of a 2048-token sequence with 60% masked, E4M3 head next
        dict(name="norm_step_e4m3", op="norm", rows=1229, src=2048, d=4096, dtype="bf16", residual=True, gather=True,
             store_sum=False, store_out=False, code="e4m3"),
        # every row of a 32768-token sequence inside the network: the residual stream is kept, an E4M3 product next
        dict(name="norm_long_all", op="norm", rows=32768, src=32768, d=4096, dtype="bf16", residual=True, gather=False,
             store_sum=True, store_out=True, code="e4m3"),
        # an fp32 model with an odd width: nothing is aligned
        dict(name="norm_odd_f32", op="norm", rows=777, src=777, d=1021, dtype="f32", residual=True, gather=False,
             store_sum=True, store_out=True, code=""),
        # the last 20 masked rows: the weight codes are streamed once
        dict(name="int8_few", op="int8", rows=20, src=4096, d=3584, V=152064, out="bf16", from_h=True),
        # one denoising step, codes in hand (the norm's)
        dict(name="int8_step", op="int8", rows=1229, src=0, d=4096, V=126464, out="bf16", from_h=False),
        # one chunk of 4096 rows of a long sequence, from the hidden states
        dict(name="int8_chunk", op="int8", rows=4096, src=32768, d=4096, V=126464, out="bf16", from_h=True),
        # a small projection with ragged sizes and fp32 results
        dict(name="int8_odd_f32", op="int8", rows=77, src=0, d=1040, V=1021, out="f32", from_h=False),
        # evaluation of the last 20 masked rows: the loss alone, few long rows
        dict(name="distill_few_loss", op="distill", rows=20, V=152064, K=32, dtype="bf16", T=1.0, mode="loss"),
        # a training step on one sequence's 1229 masked rows: loss and gradient
        dict(name="distill_step_both", op="distill", rows=1229, V=126464, K=64, dtype="bf16", T=2.0, mode="both"),
        # a chunk of 4096 masked rows: the gradient from the saved statistics, upstream gradient in hand
        dict(name="distill_chunk_grad", op="distill", rows=4096, V=126464, K=128, dtype="bf16", T=1.0, mode="grad"),
        # fp32 logits over a small odd vocabulary
        dict(name="distill_odd_f32", op="distill", rows=333, V=5003, K=17, dtype="f32", T=1.5, mode="both"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "int8", "distill"])
    if op == "norm":
        d = _log(rng, 64, 8192)
        if rng.random() < 0.75:   # most widths are multiples of 64, some are anything
            d = max(64, d // 64 * 64)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        rows = _log(rng, 1, min(32768, 32768 * 4096 // d // (2 if dtype == "f32" else 1)))
        gather = rng.random() < 0.5
        code = rng.choice(["", "int8", "e4m3"])
        return dict(op="norm", rows=rows, src=rows * 2 if gather else rows, d=d, dtype=dtype, residual=rng.random() < 0.7,
                    gather=gather, store_sum=rng.random() < 0.5, store_out=code == "" or rng.random() < 0.5, code=code)
    if op == "int8":
        d = _log(rng, 64, 8192)
        step = rng.choice([128, 128, 16, 1])
        d = max(step, d // step * step)
        V = _log(rng, 500, 152064)
        rows = _log(rng, 1, min(4096, 4096 * 126464 * 4096 // (V * d), 4096 * 126464 // V))
        from_h = d % 8 == 0 and rng.random() < 0.5
        return dict(op="int8", rows=rows, src=rows * 2 if from_h else 0, d=d, V=V,
                    out="bf16" if from_h else rng.choice(["bf16", "f32"]), from_h=from_h)
    V = _log(rng, 500, 152064)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    rows = _log(rng, 1, min(8192, 4096 * 126464 // V // (2 if dtype == "f32" else 1)))
    return dict(op="distill", rows=rows, V=V, K=_log(rng, 1, min(256, V)), dtype=dtype,
                T=rng.choice([0.7, 1.0, 2.0, 4.0]), mode=rng.choice(["loss", "grad", "both"]))


def _esize(t):
    return 4 if t == "f32" else 2


def work(case):
    n = case["rows"]
    if case["op"] == "norm":
        d, es = case["d"], _esize(case["dtype"])
        streams = 1 + case["residual"] + case["store_sum"] + case["store_out"]
        code = n * d + 4 * n if case["code"] else 0
        return {"bytes": streams * n * d * es + d * es + code + (4 * n if case["gather"] else 0), "flops": 8 * n * d}
    if case["op"] == "int8":
        d, V = case["d"], case["V"]
        rows_in = n * d * 2 + 4 * n if case["from_h"] else n * d + 4 * n
        return {"bytes": rows_in + V * d + 4 * V + n * V * _esize(case["out"]), "flops": 2 * n * V * d}
    V, K, es = case["V"], case["K"], _esize(case["dtype"])
    passes = 1 if case["mode"] == "loss" else 2
    return {"bytes": passes * n * V * es + n * K * 8 + n * 16, "flops": (3 if case["mode"] == "loss" else 6) * n * V}


# ------------------------------------------------------------------------ inputs ---

def _rows(g, src, n):
    """n of src positions, ascending, as the compaction lists them."""
    return torch.randperm(src, generator=g, device="cuda")[:n].sort().values.to(torch.int32)


def _int8_rows(x):
    """INT8 codes and row scales of fp32 rows."""
    amax = x.abs().amax(dim=1)
    inv = torch.where(amax > 0, _INT8_MAX / amax, torch.zeros_like(amax))
    return torch.round(x * inv[:, None]).to(torch.int8), amax / _INT8_MAX


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    n = case["rows"]
    s = {"case": case}
    if case["op"] == "norm":
        d, t = case["d"], _TYPES[case["dtype"]]
        # a layer's output and the residual stream, whose channels differ in size as trained ones do
        s["x"] = normal(case["src"], d).to(t)
        s["r"] = (normal(case["src"], d) * torch.exp(normal(d, std=0.7))).to(t) if case["residual"] else None
        s["gain"] = (1.0 + normal(d, std=0.2)).to(t)
        s["idx"] = _rows(g, case["src"], n) if case["gather"] else None
    elif case["op"] == "int8":
        d, V = case["d"], case["V"]
        s["wq"] = torch.empty((V, d), dtype=torch.int8, device="cuda")
        s["ws"] = torch.empty(V, dtype=torch.float32, device="cuda")
        for v in range(0, V, 32768):   # the weight's codes, laid out once
            s["wq"][v:v + 32768], s["ws"][v:v + 32768] = _int8_rows(normal(min(32768, V - v), d, std=0.02))
        if case["from_h"]:
            s["h"] = normal(case["src"], d).to(torch.bfloat16)
            s["idx"] = _rows(g, case["src"], n)
        else:
            s["hq"], s["hs"] = _int8_rows(normal(n, d))
    else:
        V, K, t = case["V"], case["K"], _TYPES[case["dtype"]]
        s["z"] = torch.empty((n, V), dtype=t, device="cuda")
        s["t"] = torch.empty((n, K), dtype=torch.float32, device="cuda")
        s["ids"] = torch.empty((n, K), dtype=torch.int32, device="cuda")
        for i in range(0, n, 512):   # a student whose logits go with its teacher's
            m = min(512, n - i)
            z = normal(m, V, std=2.0)
            top = torch.topk(z + normal(m, V), K, dim=1)
            s["z"][i:i + m], s["t"][i:i + m], s["ids"][i:i + m] = z.to(t), top.values, top.indices.to(torch.int32)
        # rows that the loss counts in full and rows of less weight
        s["g"] = torch.rand(n, generator=g, device="cuda") / n
        if case["mode"] == "grad":   # what a forward pass has kept of each row: its maximum and log-sum
            zf = [x.float() for x in s["z"].split(512)]
            s["stats"] = torch.cat([torch.stack([x.amax(1), torch.logsumexp((x - x.amax(1, keepdim=True)) / case["T"], 1)],
                                                1) for x in zf])
    return s


# -------------------------------------------------------------------- plain forms ---

def _plain_codes(y, code):
    """A row's 8-bit codes, as values, and its scale."""
    top = _INT8_MAX if code == "int8" else _E4M3_MAX
    amax = y.abs().amax(dim=1, keepdim=True)
    c = y * torch.where(amax > 0, top / amax, torch.zeros_like(amax))
    c = torch.round(c).to(torch.bfloat16) if code == "int8" else c.to(torch.float8_e4m3fn)
    return c, (amax / top)[:, 0]


def _plain_norm(s, c):
    x, r = s["x"], s["r"]
    if s["idx"] is not None:
        x = x[s["idx"].long()]
        r = r[s["idx"].long()] if r is not None else None
    v = x.float() + r.float() if r is not None else x.float()
    y = v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + 1e-6) * s["gain"].float()
    codes, scale = _plain_codes(y, c["code"]) if c["code"] else (None, None)
    return {"sum": v.to(x.dtype) if c["store_sum"] else None, "out": y.to(x.dtype) if c["store_out"] else None,
            "codes": codes, "scale": scale}


def _plain_int8(s, c):
    if c["from_h"]:
        h = s["h"][s["idx"].long()].float()
        amax = h.abs().amax(dim=1, keepdim=True)
        hs = amax / _INT8_MAX
        hq = torch.round(h * torch.where(amax > 0, _INT8_MAX / amax, torch.zeros_like(amax)))
    else:
        hq, hs = s["hq"].float(), s["hs"][:, None]
    return ((hq @ s["wq"].float().t()) * hs * s["ws"]).to(_TYPES[c["out"]])


def _plain_distill(s, c):
    T, z, ids = c["T"], s["z"].float(), s["ids"].long()
    p = torch.exp((s["t"] - s["t"].amax(dim=1, keepdim=True)) / T)
    p = p / p.sum(dim=1, keepdim=True)
    if c["mode"] == "grad":
        zmax, logsum = s["stats"][:, :1], s["stats"][:, 1:]
    else:
        zmax = z.amax(dim=1, keepdim=True)
        logsum = torch.log(torch.exp((z - zmax) / T).sum(dim=1, keepdim=True))
    loss = stats = grad = None
    if c["mode"] != "grad":
        logq = (torch.gather(z, 1, ids) - zmax) / T - logsum
        loss = T * T * (p * (torch.log(p) - logq)).sum(dim=1)
        stats = torch.cat([zmax, logsum], dim=1)
    if c["mode"] != "loss":
        grad = torch.exp((z - zmax) / T - logsum)
        grad = grad.scatter_add_(1, ids, -p)
        grad = (grad * (T * s["g"][:, None])).to(s["z"].dtype)
    return {"loss": loss, "stats": stats, "grad": grad}


# ---------------------------------------------------------------- the library's calls ---

def _own_norm(s, c):
    from mask_only_logits_amd import mosaic
    code = {"": None, "int8": mosaic.MOSAIC_INT8, "e4m3": mosaic.MOSAIC_E4M3}[c["code"]]
    sum_out, out, q, scale = mosaic.mosaic_add_rmsnorm(
        s["x"], s["gain"], eps=1e-6, residual=s["r"], row_idx=s["idx"], store_sum=c["store_sum"],
        store_out=c["store_out"], code=code)
    if c["code"]:
        q = q.to(torch.bfloat16) if c["code"] == "int8" else q.view(torch.float8_e4m3fn)
    return {"sum": sum_out, "out": out, "codes": q, "scale": scale}


def _own_int8(s, c):
    from mask_only_logits_amd import mosaic
    if c["from_h"]:
        return mosaic.mosaic_masked_logits_int8(s["h"], s["idx"], s["wq"], s["ws"])
    return mosaic.mosaic_quantized_logits(s["hq"], s["hs"], s["wq"], s["ws"], out_dtype=_TYPES[c["out"]])


def _own_distill(s, c):
    from mask_only_logits_amd import mosaic
    if c["mode"] == "grad":
        grad = mosaic.mosaic_distill_topk_grad(s["z"], s["t"], s["ids"], s["stats"], grad_loss=s["g"],
                                               temperature=c["T"])
        return {"loss": None, "stats": None, "grad": grad}
    loss, stats, grad = mosaic.mosaic_distill_topk(s["z"], s["t"], s["ids"], temperature=c["T"],
                                                   with_grad=c["mode"] == "both", grad_loss=s["g"])
    return {"loss": loss, "stats": stats, "grad": grad}


def run(state):
    c = state["case"]
    if own:
        return {"norm": _own_norm, "int8": _own_int8, "distill": _own_distill}[c["op"]](state, c)
    return {"norm": _plain_norm, "int8": _plain_int8, "distill": _plain_distill}[c["op"]](state, c)


# --------------------------------------------------------------- values in 64 bits ---

def _round_e4m3(y):
    """Nearest E4M3 value (ties to even), |y| <= 448."""
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -30))).clamp_min(-6.0)
    e = torch.where(torch.exp2(e) > y.abs().clamp_min(2.0 ** -6), e - 1, e)   # log2 next to a power of two
    e = torch.where(torch.exp2(e + 1) <= y.abs(), e + 1, e)
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    n = case["rows"]
    parts = []
    for i in range(0, n, 1024):
        rows = slice(i, min(n, i + 1024))
        if case["op"] == "norm":
            pick = s["idx"][rows].long() if s["idx"] is not None else torch.arange(rows.start, rows.stop, device="cuda")
            v = s["x"].index_select(0, pick).double()
            if s["r"] is not None:
                v = v + s["r"].index_select(0, pick).double()
            y = v / torch.sqrt(torch.square(v).sum(1, keepdim=True) / case["d"] + 1e-6) * s["gain"].double()
            codes = scale = None
            if case["code"]:
                scale = y.abs().max(dim=1).values / (_INT8_MAX if case["code"] == "int8" else _E4M3_MAX)
                unit = y / scale[:, None]
                codes = torch.round(unit) if case["code"] == "int8" else _round_e4m3(unit)
            parts.append({"sum": v if case["store_sum"] else None, "out": y if case["store_out"] else None,
                          "codes": codes, "scale": scale})
        elif case["op"] == "int8":
            if case["from_h"]:
                h = s["h"].index_select(0, s["idx"][rows].long()).double()
                hs = h.abs().max(dim=1, keepdim=True).values / _INT8_MAX
                hq = torch.round(h / hs)
            else:
                hq, hs = s["hq"][rows].double(), s["hs"][rows].double()[:, None]
            cols = [torch.mm(hq * hs, (s["wq"][v:v + 16384].double() * s["ws"][v:v + 16384].double()[:, None]).t())
                    for v in range(0, case["V"], 16384)]
            parts.append({"logits": torch.cat(cols, 1)})
        else:
            T, z, ids = case["T"], s["z"][rows].double() / case["T"], s["ids"][rows].long()
            p = torch.softmax(s["t"][rows].double() / T, dim=1)
            logq = torch.log_softmax(z, dim=1) if case["mode"] != "grad" else (
                z - s["stats"][rows, :1].double() / T - s["stats"][rows, 1:].double())
            part = {"loss": None, "stats": None, "grad": None}
            if case["mode"] != "grad":
                part["loss"] = (p * (p.log() - logq.gather(1, ids))).sum(1) * T * T
                top = z.max(1, keepdim=True).values
                part["stats"] = torch.cat([top * T, torch.logsumexp(z - top, 1, keepdim=True)], 1)
            if case["mode"] != "loss":
                target = torch.zeros_like(z).scatter_add_(1, ids, p)
                part["grad"] = T * s["g"][rows].double()[:, None] * (logq.exp() - target)
            parts.append(part)
    whole = {k: None if parts[0][k] is None else torch.cat([p[k] for p in parts]) for k in parts[0]}
    return whole["logits"] if case["op"] == "int8" else whole
