"""Cases of the layer norm, the MXFP4 head and the token log-probabilities of the masked
rows: what they are measured on.

Three operators, each with its plain form in elementary torch operations (run with
``own`` false) and as calls of this library (``own`` true):

* ``norm``   layer norm of (gathered) rows with residual addition (``mode`` fwd), and its
             backward pass with the gradients of gain and bias (``mode`` grad);
* ``fp4``    4-bit floating-point codes (E2M1) with one power-of-two scale for each 32
             elements of a row (``mode`` quant), and the matrix product of two such arrays:
             the LM head from the hidden states (``mode`` head) or from codes in hand
             (``mode`` codes);
* ``score``  log-probabilities of given tokens with the rows' entropy and top alternatives
             (``mode`` fwd), and the gradient of log-probability and entropy (``mode`` grad).

Codes are returned as the values they stand for, their scales in torch's type for 8-bit
powers of two.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------- cases ---

def listed():
    return [
        # the 20 masked rows left near the end of a denoising of a 4096-token sequence: the final norm, latency
        dict(name="norm_few_fwd", op="norm", mode="fwd", rows=20, src=4096, d=3584, dtype="bf16", residual=True,
             gather=True, store_sum=False),
        # every row of a 32768-token sequence inside the network: the residual stream is kept
        dict(name="norm_long_fwd", op="norm", mode="fwd", rows=32768, src=32768, d=4096, dtype="bf16", residual=True,
             gather=False, store_sum=True),
        # the same rows in training: the gradient of the rows, joined with the residual stream's, and of the weights
        dict(name="norm_long_grad", op="norm", mode="grad", rows=32768, src=32768, d=4096, dtype="bf16", residual=True,
             gather=False, store_sum=False),
        # an fp32 model with an odd width, in training: nothing is aligned
        dict(name="norm_odd_grad_f32", op="norm", mode="grad", rows=777, src=777, d=1021, dtype="f32", residual=False,
             gather=False, store_sum=False),
        # every hidden state of a 32768-token sequence to codes (and back, as an evaluation of the format does)
        dict(name="fp4_quant", op="fp4", mode="quant", rows=32768, src=32768, d=4096, dtype="bf16", gather=False),
        # the last 20 masked rows: the weight codes are streamed once
        dict(name="fp4_few", op="fp4", mode="head", rows=20, src=4096, d=3584, V=152064, out="bf16"),
        # one chunk of 4096 rows of a long sequence, from the hidden states
        dict(name="fp4_chunk", op="fp4", mode="head", rows=4096, src=32768, d=4096, V=126464, out="bf16"),
        # a small projection with ragged sizes and fp32 results, codes in hand
        dict(name="fp4_odd_f32", op="fp4", mode="codes", rows=77, src=0, d=1040, V=1021, out="f32"),
        # the last 20 masked rows: the sampled tokens' log-probabilities with 20 alternatives, few long rows
        dict(name="score_few_fwd", op="score", mode="fwd", rows=20, V=152064, dtype="bf16", T=1.0, top=20, entropy=True),
        # a denoising step that re-masks by entropy and margin: 1229 masked rows, the two top alternatives
        dict(name="score_step_fwd", op="score", mode="fwd", rows=1229, V=126464, dtype="bf16", T=1.0, top=2,
             entropy=True),
        # a chunk of 4096 masked rows in training: gradient of the log-probabilities and an entropy bonus
        dict(name="score_chunk_grad", op="score", mode="grad", rows=4096, V=126464, dtype="bf16", T=1.0, top=0,
             entropy=True),
        # fp32 logits over a small odd vocabulary
        dict(name="score_odd_f32", op="score", mode="fwd", rows=333, V=5003, dtype="f32", T=0.7, top=8, entropy=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "fp4", "score"])
    if op == "norm":
        d = _log(rng, 64, 16384)
        if rng.random() < 0.75:   # most widths are multiples of 64, some are anything
            d = max(64, d // 64 * 64)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        mode = rng.choice(["fwd", "grad"])
        rows = _log(rng, 1, min(32768, 32768 * 4096 // d // (2 if dtype == "f32" else 1)))
        gather = mode == "fwd" and rng.random() < 0.4
        return dict(op="norm", mode=mode, rows=rows, src=rows * 2 if gather else rows, d=d, dtype=dtype,
                    residual=rng.random() < 0.6, gather=gather, store_sum=mode == "fwd" and rng.random() < 0.5)
    if op == "fp4":
        d = _log(rng, 64, 8192)
        step = rng.choice([256, 256, 32, 1])
        d = max(step, d // step * step)
        mode = rng.choice(["quant", "head", "codes"])
        if mode == "quant":
            dtype = rng.choice(["bf16", "f32"])
            gather = rng.random() < 0.5
            rows = _log(rng, 1, min(32768, 32768 * 4096 // d // (2 if dtype == "f32" else 1)))
            return dict(op="fp4", mode=mode, rows=rows, src=rows * 2 if gather else rows, d=d, dtype=dtype,
                        gather=gather)
        V = _log(rng, 500, 152064)
        rows = _log(rng, 1, min(4096, 4096 * 126464 * 4096 // (V * d), 4096 * 126464 // V))
        return dict(op="fp4", mode=mode, rows=rows, src=rows * 2 if mode == "head" else 0, d=d, V=V,
                    out=rng.choice(["bf16", "bf16", "f32"]))
    V = _log(rng, 500, 152064)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    rows = _log(rng, 1, min(8192, 4096 * 126464 // V // (2 if dtype == "f32" else 1)))
    mode = rng.choice(["fwd", "fwd", "grad"])
    return dict(op="score", mode=mode, rows=rows, V=V, dtype=dtype, T=rng.choice([0.7, 1.0, 2.0]),
                top=rng.choice([0, 1, 2, 5, 20, 64]) if mode == "fwd" else 0, entropy=rng.random() < 0.7)


def _esize(t):
    return 4 if t == "f32" else 2


def work(case):
    n, mode = case["rows"], case["mode"]
    if case["op"] == "norm":
        d, es = case["d"], _esize(case["dtype"])
        if mode == "fwd":
            streams = 2 + case["residual"] + case["store_sum"]
            return {"bytes": streams * n * d * es + 2 * d * es + (4 * n if case["gather"] else 0), "flops": 9 * n * d}
        return {"bytes": (3 + case["residual"]) * n * d * es + 16 * n + d * es + 8 * d, "flops": 14 * n * d}
    if case["op"] == "fp4":
        d = case["d"]
        row = 17 * -(-d // 32)   # bytes of a row's codes and scales
        if mode == "quant":
            es = _esize(case["dtype"])
            return {"bytes": n * (2 * d * es + row) + (4 * n if case["gather"] else 0), "flops": 4 * n * d}
        V = case["V"]
        rows_in = n * d * 2 + 4 * n if mode == "head" else n * row
        return {"bytes": rows_in + V * row + n * V * _esize(case["out"]), "flops": 2 * n * V * d}
    V, es = case["V"], _esize(case["dtype"])
    if mode == "fwd":
        return {"bytes": n * V * es + n * (8 + 8 + 4 * case["entropy"] + 8 * case["top"]),
                "flops": (4 + 2 * case["entropy"]) * n * V}
    return {"bytes": 2 * n * V * es + n * 24, "flops": (5 + 2 * case["entropy"]) * n * V}


# ------------------------------------------------------------------------ inputs ---

def _rows(g, src, n):
    """n of src positions, ascending, as the compaction lists them."""
    return torch.randperm(src, generator=g, device="cuda")[:n].sort().values.to(torch.int32)


def _pack_fp4(x):
    """E2M1 codes, two to a byte (the even element in the low half), and scale bytes of fp32
    rows; a last, shorter block is filled up with zeros."""
    n, d = x.shape
    nb = -(-d // 32)
    b = torch.zeros((n, nb * 32), dtype=torch.float32, device=x.device)
    b[:, :d] = x
    b = b.view(n, nb, 32)
    amax = b.abs().amax(dim=2)   # (a block of zeros takes the smallest scale)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 127)
    y = (b * torch.exp2(-e.float())[:, :, None]).abs()
    # the number of midpoints that |y| has passed (a tie goes to the even code)
    c = torch.zeros(y.shape, dtype=torch.uint8, device=x.device)
    for i, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        c += (y > mid) if i % 2 == 0 else (y >= mid)
    c = (c | (torch.signbit(b).to(torch.uint8) << 3)).view(n, nb * 16, 2)
    return c[:, :, 0] | (c[:, :, 1] << 4), (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    n, mode = case["rows"], case["mode"]
    s = {"case": case}
    if case["op"] == "norm":
        d, t = case["d"], _TYPES[case["dtype"]]
        # a layer's output and the residual stream, whose channels differ in size and place as trained ones do
        wide, place = torch.exp(normal(d, std=0.7)), normal(d, std=0.5)
        s["gain"] = (1.0 + normal(d, std=0.2)).to(t)
        if mode == "fwd":
            s["x"] = normal(case["src"], d).to(t)
            s["r"] = (normal(case["src"], d) * wide + place).to(t) if case["residual"] else None
            s["bias"] = normal(d, std=0.2).to(t)
            s["idx"] = _rows(g, case["src"], n) if case["gather"] else None
        else:
            s["s"] = (normal(n, d) * wide + place).to(t)
            s["dy"] = normal(n, d, std=1e-2).to(t)
            s["dsum"] = normal(n, d, std=1e-2).to(t) if case["residual"] else None
            # what the forward pass has kept of each row: mean and reciprocal deviation
            s["stats"] = torch.empty((n, 2), dtype=torch.float64, device="cuda")
            for i in range(0, n, 4096):
                v = s["s"][i:i + 4096].double()
                s["stats"][i:i + 4096, 0] = v.mean(dim=1)
                s["stats"][i:i + 4096, 1] = torch.rsqrt(v.var(dim=1, unbiased=False) + 1e-5)
    elif case["op"] == "fp4":
        d = case["d"]
        if mode == "quant":
            s["x"] = (normal(case["src"], d) * torch.exp(normal(d, std=0.7))).to(_TYPES[case["dtype"]])
            s["idx"] = _rows(g, case["src"], n) if case["gather"] else None
            return s
        V, nb = case["V"], -(-d // 32)
        s["wq"] = torch.empty((V, nb * 16), dtype=torch.uint8, device="cuda")
        s["ws"] = torch.empty((V, nb), dtype=torch.uint8, device="cuda")
        for v in range(0, V, 32768):   # the weight's codes, laid out once
            s["wq"][v:v + 32768], s["ws"][v:v + 32768] = _pack_fp4(normal(min(32768, V - v), d, std=0.02))
        if mode == "head":
            s["h"] = normal(case["src"], d).to(torch.bfloat16)
            s["idx"] = _rows(g, case["src"], n)
        else:
            s["hq"], s["hs"] = _pack_fp4(normal(n, d))
    else:
        V, t = case["V"], _TYPES[case["dtype"]]
        s["z"] = torch.empty((n, V), dtype=t, device="cuda")
        s["tokens"] = torch.empty(n, dtype=torch.int32, device="cuda")
        for i in range(0, n, 512):   # tokens sampled from the rows' distributions, or nearly
            m = min(512, n - i)
            z = normal(m, V, std=2.0)
            noise = -torch.log(-torch.log(torch.rand(m, V, generator=g, device="cuda").clamp(1e-7, 1 - 1e-7)))
            s["z"][i:i + m], s["tokens"][i:i + m] = z.to(t), (z + noise).argmax(dim=1).to(torch.int32)
        if mode == "grad":   # what a forward pass has kept of each row: its maximum, log-sum and entropy
            s["g"] = torch.randn(n, generator=g, device="cuda") / n   # advantages
            s["h"] = (0.01 + 0.01 * torch.rand(n, generator=g, device="cuda")) / n if case["entropy"] else None
            s["stats"] = torch.empty((n, 2), dtype=torch.float32, device="cuda")
            s["ent"] = torch.empty(n, dtype=torch.float32, device="cuda")
            for i in range(0, n, 512):
                zf = s["z"][i:i + 512].double()
                m = zf.amax(1, keepdim=True)
                x = (zf - m) / case["T"]
                ls = torch.logsumexp(x, 1, keepdim=True)
                s["stats"][i:i + 512] = torch.cat([m, ls], 1)
                s["ent"][i:i + 512] = (ls - (torch.exp(x - ls) * x).sum(1, keepdim=True))[:, 0]
    return s


# -------------------------------------------------------------------- plain forms ---

def _plain_norm(s, c):
    if c["mode"] == "fwd":
        x, r = s["x"], s["r"]
        if s["idx"] is not None:
            x = x[s["idx"].long()]
            r = r[s["idx"].long()] if r is not None else None
        v = x.float() + r.float() if r is not None else x.float()
        u = v - v.mean(dim=1, keepdim=True)
        y = u * torch.rsqrt((u * u).mean(dim=1, keepdim=True) + 1e-5) * s["gain"].float() + s["bias"].float()
        return {"sum": v.to(x.dtype) if c["store_sum"] else None, "out": y.to(x.dtype)}
    mean, rstd = s["stats"][:, :1].float(), s["stats"][:, 1:].float()
    dy = s["dy"].float()
    xh = (s["s"].float() - mean) * rstd
    a = dy * s["gain"].float()
    dx = rstd * (a - a.mean(dim=1, keepdim=True) - xh * (a * xh).mean(dim=1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(s["s"].dtype), "dgain": (dy * xh).sum(dim=0), "dbias": dy.sum(dim=0)}


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _unpack_fp4(q, scale, dtype=torch.float32):
    """The values that packed codes and scale bytes stand for, [rows, 32 blocks]."""
    table = torch.tensor(_E2M1, dtype=dtype, device=q.device)
    v = torch.stack([table[(q & 15).int()], table[(q >> 4).int()]], dim=2)
    return (v.view(q.shape[0], -1, 32) * torch.exp2(scale.to(dtype) - 127.0)[:, :, None]).view(q.shape[0], -1)


def _plain_codes(x):
    """The values that the codes of fp32 rows stand for, and the scales."""
    n, d = x.shape
    nb = -(-d // 32)
    b = torch.zeros((n, nb * 32), dtype=torch.float32, device=x.device)
    b[:, :d] = x
    b = b.view(n, nb, 32)
    amax = b.abs().amax(dim=2)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 127).float()
    y = b * torch.exp2(-e)[:, :, None]
    step = torch.where(y.abs() < 2.0, 0.5, torch.where(y.abs() < 4.0, 1.0, 2.0))
    v = (torch.round(y / step) * step).clamp(-6.0, 6.0)
    return (v * torch.exp2(e)[:, :, None]).view(n, -1)[:, :d], torch.exp2(e)


def _plain_fp4(s, c):
    if c["mode"] == "quant":
        x = s["x"] if s["idx"] is None else s["x"][s["idx"].long()]
        v, scale = _plain_codes(x.float())
        return {"values": v.to(x.dtype), "scale": scale.to(torch.float8_e8m0fnu)}
    d = c["d"]
    h = _plain_codes(s["h"][s["idx"].long()].float())[0] if c["mode"] == "head" else _unpack_fp4(s["hq"], s["hs"])[:, :d]
    return (h @ _unpack_fp4(s["wq"], s["ws"])[:, :d].t()).to(_TYPES[c["out"]])


def _plain_score(s, c):
    T, z, t = c["T"], s["z"].float(), s["tokens"].long()[:, None]
    if c["mode"] == "grad":
        x = (z - s["stats"][:, :1]) / T - s["stats"][:, 1:]
        p = torch.exp(x)
        grad = p * -s["g"][:, None]
        grad = grad.scatter_add_(1, t, s["g"][:, None])
        if s["h"] is not None:
            grad = grad - s["h"][:, None] * p * (x + s["ent"][:, None])
        return {"grad": (grad / T).to(s["z"].dtype)}
    m = z.amax(dim=1, keepdim=True)
    x = (z - m) / T
    e = torch.exp(x)
    total = e.sum(dim=1, keepdim=True)
    l = torch.log(total)
    out = {"logprob": (torch.gather(x, 1, t) - l)[:, 0], "stats": torch.cat([m, l], dim=1),
           "entropy": (l - (e * x).sum(dim=1, keepdim=True) / total)[:, 0] if c["entropy"] else None}
    if c["top"]:
        # the order of the values (integers that compare as they do), then the lower index first
        b = (z + 0.0).view(torch.int32)
        b = (b ^ ((b >> 31) & 0x7fffffff)).long()
        key = (b << 32) | torch.arange(c["V"] - 1, -1, -1, device=z.device)
        ids = c["V"] - 1 - (torch.topk(key, c["top"], dim=1).values & 0xffffffff)
        out["top_ids"], out["top_logprobs"] = ids.to(torch.int32), torch.gather(x, 1, ids) - l
    return out


# ---------------------------------------------------------------- the library's calls ---

def _own_norm(s, c):
    from mask_only_logits_amd import mosaic
    if c["mode"] == "fwd":
        sum_out, out, _ = mosaic.mosaic_add_layernorm(s["x"], s["gain"], s["bias"], eps=1e-5, residual=s["r"],
                                                      row_idx=s["idx"], store_sum=c["store_sum"])
        return {"sum": sum_out, "out": out}
    dx, dgain, dbias = mosaic.mosaic_layernorm_grad(s["dy"], s["s"], s["stats"], s["gain"], grad_sum=s["dsum"])
    return {"dx": dx, "dgain": dgain, "dbias": dbias}


def _own_fp4(s, c):
    from mask_only_logits_amd import mosaic
    if c["mode"] == "quant":
        _, scale, values = mosaic.mosaic_quantize_rows_mxfp4(s["x"], row_idx=s["idx"], with_values=True)
        return {"values": values, "scale": scale.view(torch.float8_e8m0fnu)}
    t = _TYPES[c["out"]]
    if c["mode"] == "head":
        return mosaic.mosaic_masked_logits_mxfp4(s["h"], s["idx"], s["wq"], s["ws"], out_dtype=t)
    return mosaic.mosaic_quantized_logits_mxfp4(s["hq"], s["hs"], s["wq"], s["ws"], out_dtype=t)


def _own_score(s, c):
    from mask_only_logits_amd import mosaic
    if c["mode"] == "grad":
        return {"grad": mosaic.mosaic_token_logprobs_grad(s["z"], s["tokens"], s["stats"], s["g"], entropy=s["ent"],
                                                          grad_entropy=s["h"], temperature=c["T"])}
    logprob, entropy, ids, top, stats = mosaic.mosaic_token_logprobs(s["z"], s["tokens"], temperature=c["T"],
                                                                     top_n=c["top"], with_entropy=c["entropy"])
    out = {"logprob": logprob, "stats": stats, "entropy": entropy}
    if c["top"]:
        out["top_ids"], out["top_logprobs"] = ids, top
    return out


def run(state):
    c = state["case"]
    if own:
        return {"norm": _own_norm, "fp4": _own_fp4, "score": _own_score}[c["op"]](state, c)
    return {"norm": _plain_norm, "fp4": _plain_fp4, "score": _plain_score}[c["op"]](state, c)


# --------------------------------------------------------------- values in 64 bits ---

def _exact_codes(x):
    """Nearest E2M1 values in units of each block's scale, that is 2^(floor(log2 max) - 2)."""
    n, d = x.shape
    x = torch.nn.functional.pad(x, (0, -d % 32)).unflatten(1, (-1, 32))
    top = x.abs().max(dim=2, keepdim=True).values
    _, e = torch.frexp(top)
    scale = torch.ldexp(torch.ones_like(top), torch.where(top > 0, e - 3, -127).clamp(-127, 127))
    grid = torch.tensor(_E2M1[:8], dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    y = x.abs() / scale
    up, down = torch.bucketize(y, mid, right=True), torch.bucketize(y, mid)   # differ at a tie: the even one
    code = torch.where(up % 2 == 0, up, down)
    return (torch.sign(x) * grid[code] * scale).flatten(1)[:, :d], scale[:, :, 0]


def exact(case, seed):
    s = prepare(case, seed)
    n, op, mode = case["rows"], case["op"], case["mode"]
    if op == "fp4" and mode != "quant":
        w = s["wq"], s["ws"]
    parts, sums = [], []
    for i in range(0, n, 1024):
        rows = slice(i, min(n, i + 1024))
        if op == "norm" and mode == "fwd":
            pick = s["idx"][rows].long() if s["idx"] is not None else torch.arange(rows.start, rows.stop, device="cuda")
            v = s["x"].index_select(0, pick).double()
            if s["r"] is not None:
                v = v + s["r"].index_select(0, pick).double()
            var, mean = torch.var_mean(v, dim=1, unbiased=False, keepdim=True)
            y = (v - mean) / torch.sqrt(var + 1e-5)
            parts.append({"sum": v if case["store_sum"] else None,
                          "out": torch.addcmul(s["bias"].double(), y, s["gain"].double())})
        elif op == "norm":
            mean, rstd = s["stats"][rows, :1], s["stats"][rows, 1:]
            xh, dy, d = (s["s"][rows].double() - mean) * rstd, s["dy"][rows].double(), case["d"]
            a = dy * s["gain"].double()
            dx = (a - a.sum(1, keepdim=True) / d - xh * (torch.mul(a, xh).sum(1, keepdim=True) / d)) * rstd
            if s["dsum"] is not None:
                dx += s["dsum"][rows].double()
            parts.append({"dx": dx})
            sums.append((torch.mul(dy, xh).sum(0), dy.sum(0)))
        elif op == "fp4" and mode == "quant":
            x = s["x"].index_select(0, s["idx"][rows].long()) if s["idx"] is not None else s["x"][rows]
            v, scale = _exact_codes(x.double())
            parts.append({"values": v, "scale": scale})
        elif op == "fp4":
            d = case["d"]
            if mode == "head":
                h = _exact_codes(s["h"].index_select(0, s["idx"][rows].long()).double())[0]
            else:
                h = _unpack_fp4(s["hq"][rows], s["hs"][rows], torch.float64)[:, :d]
            cols = [torch.mm(h, _unpack_fp4(w[0][v:v + 16384], w[1][v:v + 16384], torch.float64)[:, :d].t())
                    for v in range(0, case["V"], 16384)]
            parts.append({"logits": torch.cat(cols, 1)})
        else:
            T, z, t = case["T"], s["z"][rows].double(), s["tokens"][rows].long()[:, None]
            if mode == "grad":
                logp = (z - s["stats"][rows, :1].double()) / T - s["stats"][rows, 1:].double()
                p = logp.exp()
                grad = torch.zeros_like(p).scatter_(1, t, 1.0).sub_(p) * s["g"][rows].double()[:, None]
                if s["h"] is not None:
                    grad -= s["h"][rows].double()[:, None] * (logp + s["ent"][rows].double()[:, None]) * p
                parts.append({"grad": grad / T})
                continue
            m = z.max(1, keepdim=True).values
            logp = torch.log_softmax(z / T, dim=1)
            part = {"logprob": logp.gather(1, t)[:, 0],
                    "stats": torch.cat([m, torch.logsumexp((z - m) / T, 1, keepdim=True)], 1),
                    "entropy": -(logp * logp.exp()).sum(1) if case["entropy"] else None}
            if case["top"]:   # the ids are whole numbers: the plain form's are compared with
                part["top_ids"] = None
                part["top_logprobs"] = torch.sort(logp, dim=1, descending=True).values[:, :case["top"]].clone()
            parts.append(part)
    whole = {k: None if parts[0][k] is None else torch.cat([p[k] for p in parts]) for k in parts[0]}
    if sums:
        whole["dgain"], whole["dbias"] = (torch.stack(v).sum(0) for v in zip(*sums))
    return whole["logits"] if op == "fp4" and mode != "quant" else whole
