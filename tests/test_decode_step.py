"""The operators around the projections used together, as one decode step of
a beam search runs them: norm -> projection -> adapters -> norm -> LM head and
beam selection -> states in their new places.  Also captured into graphs, on
other streams, between guard bands, and at offsets beyond 32 bits."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from parity_util import TOL_FP32, dev, host

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-6


class Step:
    """Buffers of a small model: hidden width D, vocabulary V, `batch` requests
    of `beams` beams, three adapters."""

    def __init__(self, q, batch=2, beams=3, D=256, V=2000, seed=90):
        self.q, self.batch, self.beams, self.V = q, batch, beams, V
        M = batch * beams
        self.W = wl.weight(seed, 0, "o", D, D, 0.05)
        self.head = wl.weight(seed, 0, "lm_head", D, V, 0.1)
        Wd = dev(self.W)
        self.s, self.z = q.group_params(Wd, 4, 64, F16)
        self.packed = q.pack_int4(Wd, self.s, self.z)
        self.headd = dev(self.head)
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.A, self.B = (r(3, 16, D) / 16).half(), (r(3, D, 16) / 4).half()
        self.w1, self.w2 = (1 + 0.1 * r(D)).half(), (1 + 0.1 * r(D)).half()
        self.start = torch.arange(0, M + 1, beams, dtype=torch.int32, device="cuda")
        self.adapter = torch.tensor([2, -1], dtype=torch.int32, device="cuda")
        self.x, self.res = r(M, D), r(M, D)
        self.scores = torch.sort(-torch.rand((batch, beams), generator=g, device="cuda"), descending=True).values
        self.finished = torch.zeros((batch, beams), dtype=torch.uint8, device="cuda")
        self.history = torch.randint(0, V, (M, 40), generator=g, device="cuda", dtype=torch.int32)
        self.cache = r(M, 4, 32, 16).to(BF16)
        self.h, self.y, self.h2 = (torch.empty((M, D), device="cuda") for _ in range(3))

    def run(self):
        q = self.q
        q.add_rmsnorm(self.x, self.w1, EPS, residual=self.res, out=self.h)
        q.matmul_q(self.h, self.packed, self.s, self.z, 4, 64, q.BC_MODE_PACKED, y=self.y)
        self.y0 = self.y.clone()
        q.lora_add(self.h, self.A, self.B, self.y, self.start, self.adapter)
        q.add_rmsnorm(self.y, self.w2, EPS, residual=self.res, out=self.h2)
        self.out = q.matmul_q_beam(self.h2, self.headd, None, None, 16, 64, q.BC_MODE_RUNTIME, self.scores,
                                   self.beams, finished=self.finished, eos=7, pad=0)
        q.beam_reorder([self.history[:, :33], self.cache[:, :, :20]], self.out[1])
        return self.out


def _norm(x, w):
    v = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    return v * w.double()


def test_step(cuda_lib):
    st = Step(cuda_lib)
    x, res, history, cache = (t.clone() for t in (st.x, st.res, st.history, st.cache))
    out = st.run()
    M = x.shape[0]
    # each operator's output from what it was given, in 64 bits
    hidden = x.double() + res.double()
    assert bool(((st.h.double() - _norm(hidden, st.w1)).abs() <= 2e-6 * _norm(hidden, st.w1).abs() + 1e-12).all())
    ref = oracle.matmul_q(host(st.h), st.W, 4, 64, "packed")
    assert (np.abs(host(st.y0) - ref["y"]) <= TOL_FP32 * ref["A"]).all()
    delta = (st.h[:3].double() @ st.A[2].double().T) @ st.B[2].double().T
    size = (st.h[:3].double().abs() @ st.A[2].double().abs().T) @ st.B[2].double().abs().T
    assert bool(((st.y[:3].double() - st.y0[:3].double() - delta).abs() <= 2e-5 * size + 2.0 ** -24 * st.y[:3].abs()).all())
    assert torch.equal(st.y[3:], st.y0[3:])                   # a request without an adapter
    second = hidden.float().double() + st.y.double()          # the residual was rounded to fp32 between the norms
    assert bool(((st.h2.double() - _norm(second, st.w2)).abs() <= 2e-6 * _norm(second, st.w2).abs() + 1e-12).all())
    logits = oracle.matmul_q(host(st.h2), st.head, 16, 64, "runtime")
    lse = np.log(np.exp(logits["y"] - logits["y"].max(1, keepdims=True)).sum(1, keepdims=True)) + logits["y"].max(1, keepdims=True)
    total = (host(st.scores).astype(np.float64).reshape(-1, 1) + logits["y"] - lse).reshape(st.batch, -1)
    slack = 2 * TOL_FP32 * logits["A"].max()                  # the projection's bar, in a logit and in the sum
    score, parent, token, ended = (host(t) for t in out)
    for b in range(st.batch):
        best = np.sort(total[b])[::-1][:st.beams]
        mine = total[b][parent[b] * st.V + token[b]]
        assert (np.abs(score[b] - best) <= slack + 1e-5).all() and (np.abs(mine - best) <= 2 * slack).all()
    assert (ended.astype(bool) == (token == 7)).all()
    at = (out[1].long() + st.beams * torch.arange(st.batch, device="cuda")[:, None]).view(-1)
    assert torch.equal(st.history[:, :33], history[at][:, :33]) and torch.equal(st.history[:, 33:], history[:, 33:])
    assert torch.equal(st.cache[:, :, :20], cache[at][:, :, :20]) and torch.equal(st.cache[:, :, 20:], cache[:, :, 20:])
    assert M == st.batch * st.beams


def test_step_captured_and_replayed(cuda_lib):
    """A captured step gives the eager step's bits, also on later inputs."""
    a, b = Step(cuda_lib), Step(cuda_lib)
    a.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = b.run()
    for i in range(3):
        x = torch.randn_like(a.x)
        for s in (a, b):
            s.x.copy_(x)
            if i == 0:
                s.res.fill_(0.5)
                s.history.copy_(torch.arange(s.history.numel(), device="cuda").view_as(s.history))
                s.cache.fill_(1.0)
        want = a.run()
        graph.replay()
        torch.cuda.synchronize()
        for p, r in zip(captured, want):
            assert torch.equal(p, r)
        assert torch.equal(a.y, b.y) and torch.equal(a.res, b.res)
        assert torch.equal(a.history, b.history) and torch.equal(a.cache, b.cache)


def test_two_graphs_share_scratch(cuda_lib):
    """Scratch holds nothing from call to call: two captured calls on one
    workspace, replayed in turn, give what each gives alone."""
    q = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(4)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    graphs = []
    for M, V in ((5, 3000), (40, 700)):
        logits = torch.randn((M, V), generator=g, device="cuda")
        scores = -torch.rand((M, 1), generator=g, device="cuda")
        x, A, B = (torch.randn(s, generator=g, device="cuda") for s in ((M, 128), (4, 8, 128), (4, 96, 8)))
        A, B, y = A.half(), B.half(), torch.zeros((M, 96), device="cuda")
        start = torch.arange(M + 1, dtype=torch.int32, device="cuda")
        ad = torch.arange(M, dtype=torch.int32, device="cuda") % 4
        outs = q.beam_select(logits, scores, 3)
        once = y.clone()
        q.lora_add(x, A, B, once, start, ad)
        mine = [torch.empty_like(t) for t in outs]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y.zero_()
            q.beam_select(logits, scores, 3, out=mine, workspace=ws)
            q.lora_add(x, A, B, y, start, ad, workspace=ws)
        graphs.append((graph, mine, outs, y, once, (logits, scores, x, A, B, start, ad)))    # what a graph reads lives on
    for _ in range(3):
        for graph, *_ in graphs:
            ws.fill_(0xA5)
            graph.replay()
    torch.cuda.synchronize()
    for _, mine, outs, y, once, _ in graphs:
        assert all(torch.equal(p, r) for p, r in zip(mine, outs)) and torch.equal(y, once)


def test_other_streams_at_once(cuda_lib):
    """The same calls on several streams at the same time, each with scratch of
    its own, given by the stream argument."""
    q = cuda_lib
    torch.manual_seed(1)
    logits, scores = torch.randn((8, 60000), device="cuda"), -torch.rand((2, 4), device="cuda")
    x, w = torch.randn((64, 2048), device="cuda"), torch.randn(2048, device="cuda")
    A, B = torch.randn((6, 32, 2048), device="cuda").to(BF16), torch.randn((6, 500, 32), device="cuda").to(BF16)
    start = torch.arange(65, dtype=torch.int32, device="cuda")
    ad = torch.arange(64, dtype=torch.int32, device="cuda") % 7 - 1
    ys = [torch.zeros((64, 500), device="cuda") for _ in range(5)]
    want_b, want_n = q.beam_select(logits, scores, 8), q.add_rmsnorm(x, w)
    q.lora_add(x, A, B, ys[4], start, ad)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for i, s in enumerate(streams):
        got.append((q.beam_select(logits, scores, 8, stream=s), q.add_rmsnorm(x, w, stream=s),
                    q.lora_add(x, A, B, ys[i], start, ad, stream=s), q.add_rmsnorm_q8(x, w, stream=s)))
    torch.cuda.synchronize()
    for b, n, y, q8 in got:
        assert all(torch.equal(p, r) for p, r in zip(b, want_b))
        assert torch.equal(n, want_n) and torch.equal(y, ys[4])
        assert all(torch.equal(p, r) for p, r in zip(q8, got[0][3]))


def _guarded(shape, dtype):
    n = int(np.prod(shape))
    buf = torch.full((n * torch.empty((), dtype=dtype).element_size() + 2048,), 0x5B, dtype=torch.uint8, device="cuda")
    return buf[1024:-1024].view(dtype).view(shape), buf


@pytest.mark.parametrize("M,S,N,R,xt", [(3, 3, 130, 16, F32), (300, 4, 131, 64, BF16), (256, 256, 36, 128, BF16), (900, 2, 64, 8, F32)])
def test_adapter_writes_stay_inside(cuda_lib, M, S, N, R, xt):
    K = 192
    x, A, B = torch.randn((M, K), device="cuda").to(xt), torch.randn((2, R, K), device="cuda").half(), torch.randn((2, N, R), device="cuda").half()
    y, ybuf = _guarded((M, N), F32)
    y.zero_()
    start = torch.tensor([i * M // S for i in range(S + 1)], dtype=torch.int32, device="cuda")
    ad = torch.arange(S, dtype=torch.int32, device="cuda") % 2
    d = cuda_lib.make_lora_descs([(x, A, B, y)])
    ws, wbuf = _guarded((cuda_lib.workspace_size_lora(d, S),), torch.uint8)
    cuda_lib.lora_add_batched(d, start, ad, workspace=ws)
    for b in (ybuf, wbuf):
        assert bool((b[:1024] == 0x5B).all()) and bool((b[-1024:] == 0x5B).all())
    assert bool(torch.isfinite(y).all()) and bool((y != 0).any(dim=1).all())


def test_norm_writes_stay_inside(cuda_lib):
    for M, D in ((3, 64), (5, 200), (2, 1003), (1, 4096), (1, 17000)):
        x = torch.randn((M, D), device="cuda")
        for ot in (F32, BF16):
            out, buf = _guarded((M, D), ot)
            res, rbuf = _guarded((M, D), ot)
            res.zero_()
            cuda_lib.add_rmsnorm(x, None, residual=res, out=out)
            for b in (buf, rbuf):
                assert bool((b[:1024] == 0x5B).all()) and bool((b[-1024:] == 0x5B).all())
        if D % 64 == 0:
            parts = [_guarded(s, d) for s, d in (((M, D), torch.uint8), ((M, D // 64), F16), ((M, D // 64), F16))]
            cuda_lib.add_rmsnorm_q8(x, None, codes=parts[0][0], scales=parts[1][0], zeros=parts[2][0])
            for _, b in parts:
                assert bool((b[:1024] == 0x5B).all()) and bool((b[-1024:] == 0x5B).all())


def test_reorder_writes_stay_inside(cuda_lib):
    for shape, cut in (((6, 3, 50), 37), ((6, 1, 4096), 4096), ((6, 5, 33), 32)):
        t, buf = _guarded(shape, torch.uint8)
        t.copy_(torch.arange(t.numel(), device="cuda").view(shape) % 251)
        old = t.clone()
        cuda_lib.beam_reorder([t[:, :, :cut]], torch.tensor([[2, 0, 1], [1, 1, 1]], dtype=torch.int32, device="cuda"))
        assert bool((buf[:1024] == 0x5B).all()) and bool((buf[-1024:] == 0x5B).all())
        assert torch.equal(t[:, :, :cut], old[[2, 0, 1, 4, 4, 4]][:, :, :cut]) and torch.equal(t[:, :, cut:], old[:, :, cut:])


def test_places_beyond_32_bits(cuda_lib):
    """More than 2^31 elements, the last of them checked."""
    q = cuda_lib
    M, N, K, R = 180000, 12288, 64, 8                        # y: 2.2e9 values
    x, A, B = torch.randn((M, K), device="cuda"), torch.randn((1, R, K), device="cuda").half(), torch.randn((1, N, R), device="cuda").half()
    y = torch.zeros((M, N), device="cuda")
    q.lora_add(x, A, B, y, torch.tensor([0, M], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))
    for r in (slice(0, 3), slice(M // 2, M // 2 + 3), slice(M - 3, M)):
        want = (x[r].double() @ A[0].double().T) @ B[0].double().T
        size = (x[r].double().abs() @ A[0].double().abs().T) @ B[0].double().abs().T
        assert bool(((y[r].double() - want).abs() <= 2e-5 * size).all())
    del x, A, B
    out = q.add_rmsnorm(y, None, out_dtype=BF16)              # 2.2e9 values in, as many out
    v = y[-2:].double() / torch.sqrt((y[-2:].double() ** 2).mean(-1, keepdim=True) + EPS)
    assert bool(((out[-2:].double() - v).abs() <= 2.0 ** -8 * v.abs() + 1e-6).all())
    del out
    # beam selection: logits are y's values
    V, batch = 151936, 14200                                  # 2.16e9 logits
    logits = y.view(-1)[:batch * V].view(batch, V)
    got = q.beam_select(logits, torch.zeros((batch, 1), device="cuda"), 2)
    for b in (0, batch - 1):
        top = torch.topk(logits[b].double(), 2)
        assert torch.equal(got[2][b].long(), top.indices)
    del logits, got
    # states: beams 2.9 GB apart
    t = y.view(-1).view(torch.uint8)[:8700000000].view(3, 2900000000)
    t[:, -5:] = torch.tensor([[1], [2], [3]], dtype=torch.uint8, device="cuda")
    q.beam_reorder([t[:, 2899999000:]], torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda"))
    assert t[:, -1].tolist() == [3, 1, 2]
