"""The operators around the masked rows' LM head used together: the compaction's list and its
device-side count feed the final norm, whose INT8 codes feed the head, whose logits feed the
distillation loss; eagerly, captured in a graph, and on two streams at once."""
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


class Step:
    """A student's step over one sequence with buffers of its own, sized for L masked rows."""

    def __init__(self, m, seed, L=300, d=512, V=1500, K=16, out_dtype=BF):
        g = torch.Generator().manual_seed(seed)
        self.m, self.L, self.d, self.V, self.K = m, L, d, V, K
        self.x = torch.randn(L, d, generator=g).to(BF).to(DEV)
        self.r = torch.randn(L, d, generator=g).to(BF).to(DEV)
        self.gain = (1 + 0.1 * torch.randn(d, generator=g)).to(BF).to(DEV)
        W = (0.05 * torch.randn(V, d, generator=g)).to(BF).to(DEV)
        self.wq, self.ws = m.mosaic_quantize_rows_int8(W)
        self.t = (2 * torch.randn(L, K, generator=g)).to(DEV)
        self.ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(L)]).to(torch.int32).to(DEV)
        self.tokens = torch.zeros(L, dtype=torch.int32, device=DEV)
        self.idx = torch.zeros(L, dtype=torch.int32, device=DEV)
        self.count = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.q = torch.zeros(L, d, dtype=torch.int8, device=DEV)
        self.scale = torch.zeros(L, device=DEV)
        self.logits = torch.zeros(L, V, dtype=out_dtype, device=DEV)
        self.loss = torch.zeros(L, device=DEV)
        self.stats = torch.zeros(L, 2, device=DEV)
        self.grad = torch.zeros(L, V, dtype=out_dtype, device=DEV)
        need = m.mosaic_distill_topk_workspace_bytes(L, V, K)
        self.ws_loss = torch.zeros(max(need, 16), dtype=torch.uint8, device=DEV)

    def mask(self, rows):
        self.tokens.zero_()
        self.tokens[rows] = 7

    def run(self, stream=None):
        m = self.m
        m.mosaic_mask_compact(self.tokens, 7, idx=self.idx, count=self.count, stream=stream)
        m.mosaic_add_rmsnorm(self.x, self.gain, residual=self.r, row_idx=self.idx, count=self.count, store_out=False,
                             code=m.MOSAIC_INT8, q=self.q, scale=self.scale, stream=stream)
        m.mosaic_quantized_logits(self.q, self.scale, self.wq, self.ws, count=self.count, out=self.logits,
                                  stream=stream)
        m.mosaic_distill_topk(self.logits, self.t, self.ids, temperature=2.0, count=self.count, loss=self.loss,
                              stats=self.stats, grad=self.grad, workspace=self.ws_loss, stream=stream)

    def outputs(self):
        return [t.clone() for t in (self.q, self.scale, self.logits, self.loss, self.stats, self.grad)]

    def clear(self):
        for t in (self.q, self.scale, self.logits, self.loss, self.stats, self.grad):
            t.fill_(3)


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("masked", [1, 20, 64, 65, 200, 300])
def test_step_against_the_plain_form(m, masked, out_dtype):
    s = Step(m, masked, out_dtype=out_dtype)
    rows = torch.randperm(s.L, generator=torch.Generator().manual_seed(masked))[:masked].sort().values
    s.mask(rows.to(DEV))
    s.clear()
    s.run()
    n = int(s.count.item())
    assert n == masked and torch.equal(s.idx[:n].cpu().long(), rows)
    _, y = plain64.norm(s.x, s.r, s.gain, 1e-6, rows)
    plain64.check_codes(s.q[:n], s.scale[:n], y, True, "codes")
    plain64.check_int8_logits(s.logits[:n], s.q[:n], s.scale[:n], s.wq, s.ws, "logits")
    plain64.check_distill(plain64.distill(s.logits[:n], s.t[:n], s.ids[:n], 2.0), s.loss[:n], s.stats[:n], s.grad[:n],
                          "loss")
    for t in s.outputs():
        assert bool((t[n:] == 3).all())


@pytest.mark.parametrize("L,V", [(300, 1500), (40, 20000)])
def test_step_captured_and_replayed(m, L, V):
    s = Step(m, 5, L=L, V=V)
    masks = [torch.randperm(L, generator=torch.Generator().manual_seed(i))[:k].to(DEV)
             for i, k in enumerate((L // 2, 0, 1, L, L - 7))]
    want = []
    for rows in masks:
        s.mask(rows)
        s.clear()
        s.run()
        want.append(s.outputs())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        s.run()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            s.run()
    torch.cuda.synchronize()
    junk = torch.randn(512, 512, device=DEV)
    for _ in range(2):
        for rows, ref in zip(masks, want):
            s.mask(rows)
            s.clear()
            junk = junk @ junk * 1e-3           # the program's own eager work in between
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(s.outputs(), ref):
                assert torch.equal(a, b)


def test_calls_that_allocate_are_captured(m):
    # outputs and workspaces taken by the calls themselves come from the graph's own memory
    s = Step(m, 6, L=24, V=40000)
    z = torch.randn(24, 40000, device=DEV).to(BF)

    def calls():
        y = m.mosaic_add_rmsnorm(s.x, s.gain, residual=s.r, store_sum=True, code=m.MOSAIC_E4M3)
        a = m.mosaic_masked_logits_int8(s.x, s.idx, s.wq, s.ws, chunk_rows=10)
        b = m.mosaic_distill_topk(z, s.t, s.ids, with_grad=True)
        c = m.mosaic_distill_topk(z, s.t, s.ids)
        return [*y, a, *b, *c[:2]]

    s.idx.copy_(torch.arange(24, dtype=torch.int32))
    want = [t.clone() for t in calls()]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = calls()
    for i in range(3):
        for t in got:
            t.fill_(1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
        calls()                                 # eager calls beside the graph


def test_steps_on_two_streams_at_once(m):
    steps = [Step(m, 1), Step(m, 2, L=40, V=30000)]
    want = []
    for s in steps:
        s.mask(torch.arange(0, s.L, 3, device=DEV))
        s.run()
        want.append(s.outputs())
        s.clear()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):
        for s, stream in zip(steps, streams):
            s.run(stream)
    torch.cuda.synchronize()
    for s, ref in zip(steps, want):
        for a, b in zip(s.outputs(), ref):
            n = int(s.count.item())
            assert torch.equal(a[:n], b[:n])


def test_norm_to_e4m3_to_the_fp8_head(m):
    s = Step(m, 9, L=200, d=512)
    _, y, q, sc = m.mosaic_add_rmsnorm(s.x, s.gain, residual=s.r, code=m.MOSAIC_E4M3)
    W = (0.05 * torch.randn(700, 512, device=DEV)).to(BF)
    wq, ws = m.mosaic_quantize_rows_fp8(W)
    got = m.mosaic_quantized_logits(q, sc, wq, ws).cpu().double()
    hv = q.cpu().view(torch.float8_e4m3fn).double() * sc.cpu().double()[:, None]
    wv = wq.cpu().view(torch.float8_e4m3fn).double() * ws.cpu().double()[:, None]
    want = hv @ wv.t()
    # 512 products summed in fp32 (at most 512 half steps of the sum of magnitudes), then bf16
    tol = want.abs() * 2.0 ** -8 + (hv.abs() @ wv.abs().t()) * 520 * 2.0 ** -24
    assert ((got - want).abs() <= tol).all()
