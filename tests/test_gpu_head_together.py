"""Layer norm, the MXFP4 head and token log-probabilities one after another, as a model's last steps use
them: in one go, captured and replayed, on other streams, and backwards."""
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


def _normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


class Step:
    """Weights, inputs and outputs of one serving step over M masked rows of L, all allocated."""

    def __init__(self, m, L, M, d, V, n, seed=0):
        self.m, self.shape = m, (L, M, d, V, n)
        self.gain, self.bias = (1 + 0.1 * _normal(seed, d)).to(BF), (0.1 * _normal(seed + 1, d)).to(BF)
        self.wq, self.ws, _ = m.mosaic_quantize_rows_mxfp4((_normal(seed + 2, V, d) * d ** -0.5).to(BF))
        self.x, self.r = torch.empty(L, d, dtype=BF, device=DEV), torch.empty(L, d, dtype=BF, device=DEV)
        self.idx = torch.empty(M, dtype=torch.int32, device=DEV)
        self.tok = torch.empty(M, dtype=torch.int32, device=DEV)
        self.y = torch.empty(M, d, dtype=BF, device=DEV)
        self.q = torch.empty_like(self.wq[:1]).expand(M, -1).contiguous()
        self.s = torch.empty(M, self.ws.shape[1], dtype=torch.uint8, device=DEV)
        self.z = torch.empty(M, V, dtype=BF, device=DEV)
        self.lp, self.H = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
        self.ids, self.top = torch.empty(M, n, dtype=torch.int32, device=DEV), torch.empty(M, n, device=DEV)
        self.st = torch.empty(M, 2, device=DEV)
        need = m.mosaic_token_logprobs_workspace_bytes(M, V, n)
        self.work = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)

    def fill(self, seed):
        L, M, d, V, _ = self.shape
        g = torch.Generator().manual_seed(seed)
        self.x.copy_(_normal(seed, L, d))
        self.r.copy_(_normal(seed + 1, L, d))
        self.idx.copy_(torch.randint(0, L, (M,), generator=g))
        self.tok.copy_(torch.randint(0, V, (M,), generator=g))

    def run(self, stream=None, work=None):
        m, n = self.m, self.shape[4]
        m.mosaic_add_layernorm(self.x, self.gain, self.bias, residual=self.r, row_idx=self.idx, out=self.y, stream=stream)
        m.mosaic_quantize_rows_mxfp4(self.y, q=self.q, scale=self.s, stream=stream)
        m.mosaic_quantized_logits_mxfp4(self.q, self.s, self.wq, self.ws, out=self.z, stream=stream)
        m.mosaic_token_logprobs(self.z, self.tok, top_n=n, logprob=self.lp, entropy=self.H, top_ids=self.ids,
                                top_logprobs=self.top, stats=self.st, workspace=self.work if work is None else work,
                                stream=stream)

    def outs(self):
        return [t.clone() for t in (self.y, self.q, self.s, self.z, self.lp, self.H, self.ids, self.top, self.st)]

    def clear(self):
        for t in (self.y, self.q, self.s, self.z, self.lp, self.H, self.ids, self.top, self.st, self.work):
            t.zero_()


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


SHAPES = [(50, 20, 512, 70001, 20), (400, 129, 1040, 33000, 2), (700, 600, 256, 5003, 64), (3, 1, 100, 40000, 5)]


@pytest.mark.parametrize("L,M,d,V,n", SHAPES)
def test_step(m, L, M, d, V, n):
    a = Step(m, L, M, d, V, n)
    a.fill(7)
    a.run()
    i = a.idx.long()
    head64.check_layernorm(a.x[i], a.r[i], a.gain, a.bias, 1e-5, None, None, a.y, None, "norm")
    q, s = head64.mxfp4_codes(a.y)
    assert torch.equal(a.q.cpu(), q) and torch.equal(a.s.cpu(), s)
    head64.check_mxfp4_logits(a.z, a.q, a.s, a.wq, a.ws, d, "logits")
    head64.check_logprobs(a.z, a.tok, 1.0, a.lp, a.H, a.ids, a.top, a.st, "log-probabilities")
    # the head from the normed rows gives the logits of the codes in hand
    z = m.mosaic_masked_logits_mxfp4(a.y, torch.arange(M, dtype=torch.int32, device=DEV), a.wq, a.ws)
    assert torch.equal(z, a.z)


@pytest.mark.parametrize("L,M,d,V,n", SHAPES)
def test_step_captured_and_replayed(m, L, M, d, V, n):
    a, b = Step(m, L, M, d, V, n), Step(m, L, M, d, V, n, seed=90)
    want = []
    for seed in range(4):
        a.fill(seed), b.fill(seed + 50)
        a.run(), b.run()
        want.append((a.outs(), b.outs()))
    # two graphs that share a workspace, replayed one after the other
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        a.run()
    with torch.cuda.graph(gb):
        b.run(work=a.work)
    for seed in (1, 3, 0, 2, 1):
        a.clear(), b.clear()
        a.fill(seed), b.fill(seed + 50)
        ga.replay()
        gb.replay()
        assert _same(a.outs(), want[seed][0]) and _same(b.outs(), want[seed][1])
        # eager work between the replays, which leaves them alone
        a.run(), b.run()
        torch.cuda.synchronize()
        assert _same(a.outs(), want[seed][0]) and _same(b.outs(), want[seed][1])


@pytest.mark.parametrize("L,M,d,V,n", SHAPES)
def test_two_steps_at_once_on_two_streams(m, L, M, d, V, n):
    both = [Step(m, L, M, d, V, n), Step(m, L, M, d, V, n, seed=90)]
    want = []
    for k, a in enumerate(both):
        a.fill(k)
        a.run()
        want.append(a.outs())
        a.clear()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, a in zip(streams, both):
            a.run(stream=s)   # not the current stream
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for a, w in zip(both, want):
        assert _same(a.outs(), w)
    # what the calls allocate themselves belongs to their stream
    for s, a, w in zip(streams, both, want):
        s.wait_stream(torch.cuda.current_stream())
        got = m.mosaic_token_logprobs(a.z, a.tok, top_n=n, with_entropy=True, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert _same(got, w[4:])
        for t in got:
            t.record_stream(torch.cuda.current_stream())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,d,V", [(40, 256, 5003), (300, 136, 999), (1, 64, 7)])
def test_training_step(m, M, d, V, dtype):
    """Norm, logits, log-probabilities with an entropy bonus, and back: each operator against 64-bit
    arithmetic on what the one before it left.  A captured step gives the same bits."""
    x, r = _normal(1, M, d).to(dtype), _normal(2, M, d).to(dtype)
    gain, bias = 1 + 0.1 * _normal(3, d), 0.1 * _normal(4, d)
    w = (_normal(5, V, d) * d ** -0.5).to(dtype)
    tok = torch.randint(0, V, (M,), generator=torch.Generator().manual_seed(6)).to(torch.int32).to(DEV)
    tok[M // 2] = -1 if M > 1 else tok[0]   # a padded row
    g, h = _normal(7, M), 0.1 * _normal(8, M)
    idx = torch.arange(M, dtype=torch.int32, device=DEV)

    def step():
        s, y, st = m.mosaic_add_layernorm(x, gain, bias, residual=r, store_sum=True, with_stats=True)
        z = m.mosaic_masked_logits(y, idx, w)
        lp, H, _, _, zs = m.mosaic_token_logprobs(z, tok, with_entropy=True, temperature=0.7)
        dz = m.mosaic_token_logprobs_grad(z, tok, zs, g, entropy=H, grad_entropy=h, temperature=0.7)
        dy = torch.mm(dz.float(), w.float()).to(dtype)
        dx, dg, db = m.mosaic_layernorm_grad(dy, s, st, gain, grad_sum=r)
        return y, s, st, z, lp, H, zs, dz, dy, dx, dg, db

    got = step()
    y, s, st, z, lp, H, zs, dz, dy, dx, dg, db = got
    head64.check_layernorm(x, r, gain, bias, 1e-5, None, s, y, st, "norm")
    head64.check_logprobs(z, tok, 0.7, lp, H, None, None, zs, "log-probabilities")
    head64.check_logprobs_grad(z, tok, 0.7, g, h, dz, "their gradient")
    head64.check_layernorm_grad(dy, s, st, gain, None, r, dx, dg, db, "the norm's")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for _ in range(3):
        for t in kept:
            t.zero_()
        graph.replay()
        assert _same(kept, got)
        step()
        torch.cuda.synchronize()


def test_gradient_of_the_run_against_differences(m):
    """fp32 all through.  With f the loss in 64 bits, f(x + e u) - f(x - e u) over 2 e is off by e^2 times a
    third derivative: for e = 1e-4 below 1e-6 of the scale of f here; the gradient's own error is a few
    hundred roundings of 2^-24, below 1e-4 of that scale."""
    M, d, V, T = 6, 96, 300, 0.9
    x, gain, bias, w = _normal(1, M, d), 1 + 0.1 * _normal(2, d), 0.1 * _normal(3, d), _normal(4, V, d) * d ** -0.5
    tok = torch.arange(M, dtype=torch.int32, device=DEV) * 7
    g, h = _normal(5, M), _normal(6, M)

    def loss(x, gain, bias):
        x, gain, bias = (t.double().cpu() for t in (x, gain, bias))
        s = x - x.mean(1, keepdim=True)
        y = s / (s.square().mean(1, keepdim=True) + float(torch.tensor(1e-5))).sqrt() * gain + bias
        logp = torch.log_softmax(y @ w.double().cpu().T / T, 1)
        lp = logp.gather(1, tok.long().cpu()[:, None])[:, 0]
        return float((g.double().cpu() * lp - h.double().cpu() * (logp.exp() * logp).sum(1)).sum())

    _, y, st = m.mosaic_add_layernorm(x, gain, bias, with_stats=True)
    z = torch.mm(y, w.T.contiguous())
    _, H, _, _, zs = m.mosaic_token_logprobs(z, tok, temperature=T, with_entropy=True)
    dz = m.mosaic_token_logprobs_grad(z, tok, zs, g, entropy=H, grad_entropy=h, temperature=T)
    dx, dg, db = m.mosaic_layernorm_grad(torch.mm(dz, w), x, st, gain)
    for k, (t, grad) in enumerate(((x, dx), (gain, dg), (bias, db))):
        u, e = _normal(20 + k, *t.shape).double(), 1e-4
        args = [x.double(), gain.double(), bias.double()]
        up, down = list(args), list(args)
        up[k], down[k] = args[k] + e * u, args[k] - e * u
        want = (loss(*up) - loss(*down)) / (2 * e)
        scale = float((grad.double() * u).abs().sum())
        assert abs(float((grad.double() * u).sum()) - want) <= 1e-4 * scale + 1e-6, (k, want)
