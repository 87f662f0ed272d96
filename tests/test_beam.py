"""Beam search: selection (bc_beam_select, bc_matmul_q_beam) and reordering of
the states (bc_beam_reorder), against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import workloads as wl
from parity_util import dev

FAKE = 0x10000                    # aligned non-null address: never dereferenced
INF = float("inf")


def _totals(logits, scores, finished, pad):
    """[batch][beams * V] in 64 bits."""
    batch, beams = scores.shape
    l = logits.astype(np.float64).reshape(batch, beams, -1)
    l = np.where(np.isnan(l), -INF, np.minimum(l, np.finfo(np.float32).max))
    m = l.max(-1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        lse = m + np.log(np.exp(l - np.where(np.isfinite(m), m, 0)).sum(-1, keepdims=True))
        s = np.where(np.isnan(scores), -INF, scores).astype(np.float64)[..., None]
        t = s + (l - lse)
    t[np.isnan(t) | np.isneginf(np.broadcast_to(s, t.shape))] = -INF
    if finished is not None:
        for b, w in zip(*np.nonzero(finished)):
            t[b, w] = -INF
            t[b, w, pad] = s[b, w, 0]
    return t.reshape(batch, -1)


def _check(got, logits, scores, n_out, finished=None, eos=-1, pad=0):
    """Places and order: those of the exact totals, except where two exact
    totals are within `near` of each other.  near: the sums of exponentials are
    sums of fp32 values each 2^-23 off (two units in the last place) with the
    differences to the maximum rounded to 2^-24 of themselves, so that
    x exp(-x) <= 1 makes that at most 2^-24 of the largest term each; a thread's
    eight values are added in fp32 (7 roundings of 2^-24)."""
    near = 2 * (2.0 ** -23 + 2.0 ** -24 + 7 * 2.0 ** -24)
    out, parent, token, ended = (t.cpu().numpy() for t in got)
    V = logits.shape[1]
    t = _totals(logits, scores, finished, pad)
    order = np.argsort(-t, axis=1, kind="stable")[:, :n_out]
    flat = parent.astype(np.int64) * V + token
    assert (token >= 0).all() and (token < V).all() and (parent >= 0).all()
    for b in range(t.shape[0]):
        assert len(set(flat[b])) == n_out
        want, mine = t[b][order[b]], t[b][flat[b]]
        same = flat[b] == order[b]
        with np.errstate(invalid="ignore"):
            assert (same | (np.abs(want - mine) <= near)).all(), (b, np.nonzero(~same))
        both = np.isfinite(want)
        assert (flat[b][~both] == order[b][~both]).all()
        assert (np.isneginf(out[b]) == ~both).all()
        # fp32 rounding of the total beside the sum's error
        assert (np.abs(out[b][both] - mine[both]) <= near + 2.0 ** -24 * np.abs(mine[both])).all()
    e = token == eos
    if finished is not None:
        e |= np.take_along_axis(finished.astype(bool), parent, 1)
    assert (ended.astype(bool) == e).all()


def _select(q, logits, scores, n_out, finished=None, **kw):
    return q.beam_select(dev(logits), dev(scores), n_out,
                         finished=None if finished is None else dev(finished), **kw)


def _draw(batch, beams, V, seed):
    rng = np.random.default_rng(seed)
    logits = (2.5 * rng.standard_normal((batch * beams, V))).astype(np.float32)
    scores = (-20 * rng.random((batch, beams))).astype(np.float32)
    return rng, logits, scores


@pytest.mark.gpu
@pytest.mark.parametrize("batch,beams,V,n_out", [
    (1, 1, 1, 1), (1, 1, 5, 5), (2, 3, 7, 6), (1, 4, 2048, 8), (3, 2, 2049, 4), (1, 4, 32003, 8),
    (2, 5, 50001, 10), (1, 32, 3001, 64), (40, 4, 1000, 4), (2, 8, 20480, 16), (1, 1, 151936, 64), (70, 1, 4099, 2)])
@pytest.mark.parametrize("finished", [False, True])
def test_select(cuda_lib, batch, beams, V, n_out, finished):
    rng, logits, scores = _draw(batch, beams, V, batch * 7 + V)
    fin = (rng.random((batch, beams)) < 0.3).astype(np.uint8) if finished else None
    eos, pad = V // 3, V - 1
    _check(_select(cuda_lib, logits, scores, n_out, fin, eos=eos, pad=pad), logits, scores, n_out, fin, eos, pad)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [0, 3, 40])
def test_every_beam_finished(cuda_lib, pad):
    _, logits, scores = _draw(2, 4, 500, pad)
    fin = np.ones((2, 4), np.uint8)
    _check(_select(cuda_lib, logits, scores, 8, fin, pad=pad), logits, scores, 8, fin, -1, pad)


@pytest.mark.gpu
def test_first_step_and_beams_without_a_score(cuda_lib):
    _, logits, scores = _draw(3, 4, 5000, 3)
    scores[:, 1:] = -INF
    scores[1] = -INF
    scores[2, 1] = np.nan
    _check(_select(cuda_lib, logits, scores, 6), logits, scores, 6)
    fin = np.array([[1, 0, 1, 0]] * 3, np.uint8)
    _check(_select(cuda_lib, logits, scores, 6, fin, pad=9), logits, scores, 6, fin, -1, 9)


@pytest.mark.gpu
def test_masked_tokens(cuda_lib):
    """Rows that leave a few tokens, one, or none; NaN; the type's lowest value."""
    rng, logits, scores = _draw(6, 2, 6000, 4)
    keep = rng.random(logits.shape) < 0.001
    logits[:4][~keep[:4]] = -INF
    logits[4] = -INF
    logits[5] = -INF
    logits[5, 4321] = 1.5
    logits[6] = -INF
    logits[7] = -INF                                 # a request with nothing at all
    logits[8, ::2] = np.nan
    logits[9] = np.finfo(np.float32).min
    logits[10, 17] = np.finfo(np.float32).max
    logits[11, 5999] = 3e38
    _check(_select(cuda_lib, logits, scores, 10), logits, scores, 10)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [300, 6000, 30000])
def test_equal_totals_go_to_the_lowest_place(cuda_lib, V):
    """Equal rows at equal scores, and rows of one value: exact ties."""
    batch, beams, n_out = 2, 4, 12
    logits = np.zeros((batch * beams, V), np.float32)
    row = np.round(np.random.default_rng(1).standard_normal(V) * 2).astype(np.float32)
    logits[beams:] = row
    scores = np.full((batch, beams), -2.0, np.float32)
    got = _select(cuda_lib, logits, scores, n_out)
    parent, token = got[1].cpu().numpy(), got[2].cpu().numpy()
    assert (parent[0] == 0).all() and (token[0] == np.arange(n_out)).all()
    t = np.concatenate([row] * beams).astype(np.float64)
    order = np.argsort(-t, kind="stable")[:n_out]
    assert (parent[1] * V + token[1] == order).all()


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["rising", "falling", "one thread"])
def test_orders_that_fill_the_candidates(cuda_lib, how):
    V, n_out = 40000, 64
    v = np.linspace(-8, 8, V).astype(np.float32)
    if how == "falling":
        v = v[::-1].copy()
    elif how == "one thread":
        v = np.full(V, -5, np.float32)
        v[256 * np.arange(V // 256) + 3] = np.linspace(0, 4, V // 256)
    logits = np.stack([v, v[::-1]])
    scores = np.array([[-1.0, -1.5]], np.float32)
    _check(_select(cuda_lib, logits, scores, n_out), logits, scores, n_out)


@pytest.mark.gpu
def test_select_unaligned_rows_and_guard(cuda_lib):
    """Logits that begin off 16 bytes; nothing is written around the outputs."""
    batch, beams, V, n_out = 2, 3, 4004, 5
    _, logits, scores = _draw(batch, beams, V, 8)
    buf = torch.empty(logits.size + 3, device="cuda")
    view = buf[3:].view(batch * beams, V)
    view.copy_(dev(logits))
    outs, bufs = [], []
    for dt in (torch.float32, torch.int32, torch.int32, torch.uint8):
        b = torch.full((batch * n_out + 32,), 77, dtype=dt, device="cuda")
        bufs.append(b)
        outs.append(b[16:16 + batch * n_out].view(batch, n_out))
    need = cuda_lib.workspace_size_beam(batch, beams, V, n_out)
    ws = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    got = cuda_lib.beam_select(view, dev(scores), n_out, out=outs, workspace=ws[256:256 + need])
    _check(got, logits, scores, n_out)
    for b in bufs:
        assert bool((b[:16] == 77).all()) and bool((b[16 + batch * n_out:] == 77).all())
    assert bool((ws[:256] == 77).all()) and bool((ws[256 + need:] == 77).all())


@pytest.mark.gpu
@pytest.mark.parametrize("mode,bits", [("packed", 4), ("runtime", 16)])
def test_head_and_selection_in_one_call(cuda_lib, mode, bits):
    batch, beams, N, K, n_out = 2, 3, 3000, 256, 6
    W = dev(wl.weight(71, 0, "lm_head", K, N, 0.2))
    x = dev(wl.activation(71, 0, "x", batch * beams, K))
    if mode == "packed":
        s, z = cuda_lib.group_params(W, 4, 64, torch.float16)
        Wk, mid = cuda_lib.pack_int4(W, s, z), cuda_lib.BC_MODE_PACKED
    else:
        s = z = None
        Wk, mid = W, cuda_lib.BC_MODE_RUNTIME
    scores = -torch.rand((batch, beams), device="cuda")
    a = cuda_lib.matmul_q_beam(x, Wk, s, z, bits, 64, mid, scores, n_out, eos=5)
    y = cuda_lib.matmul_q(x, Wk, s, z, bits, 64, mid)
    b = cuda_lib.beam_select(y, scores, n_out, eos=5)
    for p, r in zip(a, b):
        assert torch.equal(p, r)
    _check(a, y.cpu().numpy(), scores.cpu().numpy(), n_out, eos=5)


def test_select_rejects_on_host():
    import quantized_matmul_02_b200 as q
    at = [FAKE + (i << 24) for i in range(10)]
    ok = dict(logits=at[0], scores=at[1], finished=None, batch=2, beams=4, V=1000, n_out=8, eos=-1, pad=0,
              out=at[3], parent=at[4], token=at[5], ended=None, ws=at[6], wsb=1 << 20, stream=None)
    call = lambda **kw: q.lib.bc_beam_select(*{**ok, **kw}.values())  # noqa: E731
    for k in ("logits", "scores", "out", "parent", "token"):
        assert call(**{k: None}) == 1
    for k in ("batch", "beams", "V", "n_out"):
        assert call(**{k: 0}) == 1 and call(**{k: -3}) == 1
    assert call(beams=33) == 2 and call(n_out=65) == 2 and call(V=(1 << 22) + 1) == 2 and call(batch=1 << 16) == 2
    assert call(V=1 << 22, wsb=256) == 4
    assert call(V=1, n_out=5) == 1                   # fewer continuations than asked for
    assert call(finished=at[2], pad=1000) == 1 and call(finished=at[2], pad=-1) == 1
    assert call(logits=at[0] + 2) == 3 and call(ws=at[6] + 16) == 3
    assert call(wsb=256) == 4 and call(ws=None) == 4
    assert call(out=at[4]) == 1 and call(token=at[0]) == 1 and call(ended=at[6]) == 1
    assert q.workspace_size_beam(2, 4, 1000, 8) > 0 and q.workspace_size_beam(2, 33, 1000, 8) == 0
    m = [at[0], 0, at[1], None, None, 2, 4, 1000, 64, 16, 64, 0, at[2], None, 8, -1, 0, at[3], at[4], at[5], None,
         at[6], 256, None]
    assert q.lib.bc_matmul_q_beam(*m) == 4
    assert q.lib.bc_matmul_q_beam(*m[:12], None, *m[13:]) == 1
    assert q.lib.bc_matmul_q_beam(*m[:8], 96, *m[9:]) == 1
    with pytest.raises(ValueError):
        q.beam_select(torch.zeros(4, 9), torch.zeros(1, 4), 4)


def _sum_bound(row):
    """How far a row's log-sum-exp may be off.  With d a logit's distance to the
    largest one and p its probability: the difference and its product with
    log2(e) round by 2^-24 of themselves, the constant is 2^-26 off, so exp(-d)
    is (2^-23 + 2^-26) d off, and 2^-22 by the exponential's own error; both are
    weighted by p.  The largest one's term is exactly 1.  A thread's eight
    terms take 7 roundings of 2^-24, the rest is in fp64."""
    d = row.max() - row.astype(np.float64)
    e = np.exp(-d)
    p = e / e.sum()
    return 2.0 ** -22 * (1 - p.max()) + (2.0 ** -23 + 2.0 ** -26) * (p * d).sum() + 7 * 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("batch,V", [(3, 102400), (640, 20480)])       # one launch, and two
def test_near_certain_tokens(cuda_lib, batch, V):
    """Rows with one token 8 to 15.9 above the next one, which the same thread
    meets some tiles earlier, and all others 40 below: the sums are 1 and a
    little.  That little is off by the second token's own error (2^-22 and 2^-23
    + 2^-25 of its distance) and by the others, which may vanish beside 1."""
    rng = np.random.default_rng(11)
    logits = np.full((batch, V), -30.0, np.float32)
    gap = rng.uniform(8, 15.9, batch)
    first = rng.integers(0, 4096, batch)
    later = first + 4096 * rng.integers(1, 4, batch)
    top = rng.uniform(9.5, 10.5, batch).astype(np.float32)
    logits[np.arange(batch), later] = top
    logits[np.arange(batch), first] = top - gap
    out, parent, token, _ = (t.cpu().numpy() for t in _select(cuda_lib, logits, np.zeros((batch, 1), np.float32), 2))
    assert (token[:, 0] == later).all() and (token[:, 1] == first).all()
    gap = top.astype(np.float64) - logits[np.arange(batch), first]
    rest = (V - 2) * np.exp(-30.0 - top.astype(np.float64))
    want = -np.log1p(np.exp(-gap) + rest)
    bound = np.exp(-gap) * (2.0 ** -22 + gap * (2.0 ** -23 + 2.0 ** -25)) + 2 * rest
    assert (np.abs(out[:, 0] - want) <= bound + 2.0 ** -24 * np.abs(want)).all(), np.abs(out[:, 0] - want).max()
    assert (np.abs(out[:, 1] - (want - gap)) <= bound + 2.0 ** -24 * np.abs(want - gap)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("batch,V", [(3, 102400), (640, 20480)])
def test_sums_of_flat_and_spread_rows(cuda_lib, batch, V):
    """Totals of rows whose weight lies far below the largest logit, or spreads."""
    rng = np.random.default_rng(12)
    logits = np.empty((batch, V), np.float32)
    for b in range(batch):
        kind = b % 4
        if kind == 0:
            logits[b] = -rng.uniform(2, 14)          # one value, each term off the same way
            logits[b, rng.integers(0, V)] = rng.uniform(0, 1)
        elif kind == 1:
            logits[b] = rng.uniform(-20, 20, V)
        elif kind == 2:
            logits[b] = np.linspace(-12, rng.uniform(0, 12), V)         # every tile has a larger one
        else:
            logits[b] = 2.5 * rng.standard_normal(V)
    row = logits.astype(np.float64)
    top = row.max(1)
    want = -np.log(np.exp(row - top[:, None]).sum(1))
    scores = (-want).astype(np.float32)              # totals near 0, which rounding to fp32 leaves as they are
    out, _, token, _ = (t.cpu().numpy()[:, 0] for t in _select(cuda_lib, logits, scores[:, None], 1))
    assert (row[np.arange(batch), token] == top).all()
    err = np.abs(out - (scores + want))
    bound = np.array([_sum_bound(r) for r in logits])
    assert (err <= bound + 2.0 ** -24 * np.abs(scores + want)).all(), [float((err / bound)[k::4].max()) for k in range(4)]


@pytest.mark.parametrize("mode,bits", [(0, 16), (0, 3), (1, 4), (2, 5)])       # runtime, packed, ranges
def test_head_and_selection_refuse_outputs_over_what_the_matmul_reads(mode, bits):
    """x, W, scales and zeros, from their first byte and to their last."""
    import quantized_matmul_02_b200 as q
    batch, beams, N, K, n_out = 2, 4, 1000, 128, 8
    at = [FAKE + (i << 24) for i in range(12)]
    need = q.workspace_size_matmul_beam(batch, beams, N, K, n_out, mode)
    sizes = {0: batch * beams * K * 4, 1: N * K * bits // 8 if mode == 1 else N * K * 2}
    if bits != 16:
        sizes[2] = N * (K // 64) * (2 if mode == 1 else 4)
        if mode != 2:
            sizes[3] = sizes[2]

    def call(**kw):
        a = dict(x=at[0], xt=0, W=at[1], s=at[2] if 2 in sizes else None, z=at[3] if 3 in sizes else None, batch=batch,
                 beams=beams, N=N, K=K, bits=bits, group=64, mode=mode, scores=at[4], finished=None, n_out=n_out, eos=-1,
                 pad=0, out=at[5], parent=at[6], token=at[7], ended=at[8], ws=at[9], wsb=need, stream=None)
        return q.lib.bc_matmul_q_beam(*{**a, **kw}.values())

    for i, size in sizes.items():
        for name in ("out", "parent", "token", "ended"):
            assert call(**{name: at[i]}) == 1 and call(**{name: at[i] + size - 4}) == 1
        assert call(ws=at[i]) == 1 and call(ws=at[i] + (size - 1) // 256 * 256) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("batch,beams,V,n_out", [
    (2, 32, 151936, 64),        # 9 spans a beam, 288 lists a request
    (1, 32, 151936, 64),        # 18 spans, 576 lists
    (16, 8, 100000, 16),        # 4 spans
    (60, 3, 40003, 6),          # 3 spans, rows at odd places
    (3, 16, 60001, 33)])
def test_select_over_beams_of_several_spans(cuda_lib, batch, beams, V, n_out):
    rng, logits, scores = _draw(batch, beams, V, V + beams)
    scores = (0.1 * scores).astype(np.float32)          # many beams have a part in the result
    fin = (rng.random((batch, beams)) < 0.2).astype(np.uint8)
    _check(_select(cuda_lib, logits, scores, n_out), logits, scores, n_out)
    _check(_select(cuda_lib, logits, scores, n_out, fin, eos=7, pad=11), logits, scores, n_out, fin, 7, 11)


@pytest.mark.gpu
@pytest.mark.parametrize("batch,beams,V,n_out", [(1, 8, 40000, 16), (1, 8, 40000, 64), (700, 1, 60000, 8), (2, 32, 60000, 64),
                                                 (1, 32, 151936, 64)])
@pytest.mark.parametrize("values", [1, 3])
def test_equal_totals_in_long_spans_and_many_lists(cuda_lib, batch, beams, V, n_out, values):
    """More equal maxima than a list takes, in spans of more than eight tiles
    and over many lists: beams share a row and a score, so the lowest places of
    the first beam that has the best value win."""
    row = np.random.default_rng(V).integers(0, values, V).astype(np.float32)
    logits = np.broadcast_to(row, (batch * beams, V))
    scores = np.full((batch, beams), -2.0, np.float32)
    got = _select(cuda_lib, logits, scores, n_out)
    at = np.nonzero(row == values - 1)[0][:n_out]
    assert at.size == n_out
    assert (got[1].cpu().numpy() == 0).all() and (got[2].cpu().numpy() == at).all()


@pytest.mark.gpu
def test_few_best_tokens_of_every_beam(cuda_lib):
    """One token a beam stands out and the others are equal: what the beams'
    first tokens leave is filled by the lowest places of the best beam."""
    beams, V, n_out = 32, 100000, 64
    logits = np.zeros((beams, V), np.float32)
    top = 99999 - 3000 * np.arange(beams)
    logits[np.arange(beams), top] = 5.0
    scores = np.full((1, beams), -1.0, np.float32)
    out, parent, token, _ = (t.cpu().numpy()[0] for t in _select(cuda_lib, logits, scores, n_out))
    assert (np.sort(parent[:beams]) == np.arange(beams)).all() and (token[:beams] == top[parent[:beams]]).all()
    # the beams' sums agree but for their last bits, so the rest is all of one beam
    assert (parent[beams:] == parent[beams]).all() and (token[beams:] == np.arange(n_out - beams)).all()
    near = _sum_bound(logits[0])
    total = -1.0 - np.log(np.exp(logits[0].astype(np.float64)).sum())
    assert (np.abs(out - np.where(np.arange(n_out) < beams, total + 5, total)) <= near + 2.0 ** -24 * 16).all()


# ---- reordering ----
@pytest.mark.gpu
@pytest.mark.parametrize("beams", [1, 2, 4, 5, 8, 13, 32])
@pytest.mark.parametrize("shape,cut,dt", [((1,), None, torch.int32), ((3, 40, 16), 25, torch.bfloat16),
                                          ((5, 33), 17, torch.uint8), ((2, 1000, 8), 999, torch.float16),
                                          ((77,), None, torch.uint8), ((4, 6), 5, torch.int16),
                                          ((2, 1501), 1499, torch.uint8), ((9001,), None, torch.uint8),
                                          ((3, 5003), 5001, torch.int16), ((1, 20003), 20000, torch.uint8),
                                          ((2, 515), 513, torch.int32), ((512,), None, torch.uint8)])
def test_reorder(cuda_lib, beams, shape, cut, dt):
    batch = 3
    g = torch.Generator().manual_seed(beams)
    t = torch.randint(0, 250, (batch * beams, *shape), generator=g).to(dt).cuda()
    parent = torch.randint(0, beams, (batch, beams), generator=g).int().cuda()
    view = t if cut is None else t[:, :, :cut]
    want = t.clone()
    at = (parent.long() + beams * torch.arange(batch, device="cuda")[:, None]).view(-1)
    (want if cut is None else want[:, :, :cut]).copy_((t if cut is None else t[:, :, :cut])[at])
    cuda_lib.beam_reorder([view], parent)
    assert torch.equal(t, want)


@pytest.mark.gpu
def test_reorder_many_states_at_once(cuda_lib):
    """More states than one launch takes, of different sizes; parents that are
    not beams leave theirs; a view of wider parents."""
    batch, beams = 2, 4
    states = [torch.randint(0, 99, (batch * beams, 1 + i % 7, 3 + i), device="cuda", dtype=torch.int32) for i in range(70)]
    wide = torch.tensor([[3, 3, 0, 7, 1], [1, 0, -1, 2, 0]], dtype=torch.int32, device="cuda")
    eff = torch.tensor([[3, 3, 0, 3], [1, 0, 2, 2]], device="cuda")
    at = (eff + beams * torch.arange(batch, device="cuda")[:, None]).view(-1)
    want = [s[at] for s in states]
    cuda_lib.beam_reorder(states, wide[:, :beams])
    for s, w in zip(states, want):
        assert torch.equal(s, w)


@pytest.mark.gpu
def test_reorder_layers_outside_beams(cuda_lib):
    """[layers][batch * beams][...]: runs of one state that lie beams apart."""
    q, layers, beams, n = cuda_lib, 3, 4, 20
    t = torch.randn((layers, beams, n), device="cuda")
    parent = torch.tensor([[2, 2, 1, 0]], dtype=torch.int32, device="cuda")
    want = t[:, parent[0].long()]
    q.beam_reorder([t.transpose(0, 1)], parent)
    assert torch.equal(t, want)


def test_reorder_rejects_on_host():
    import quantized_matmul_02_b200 as q

    def call(state=(FAKE, 4, 64, 128, 1024), count=1, parent=FAKE + (1 << 24), stride=4, batch=2, beams=4, more=()):
        arr = (q.BeamState * max(1, 1 + len(more)))(q.BeamState(*state), *[q.BeamState(*m) for m in more])
        return q.lib.bc_beam_reorder(arr, count, parent, stride, batch, beams, None)

    assert q.lib.bc_beam_reorder(None, 1, FAKE, 4, 2, 4, None) == 1
    assert call(count=0) == 1 and call(parent=None) == 1 and call(batch=0) == 1 and call(beams=-1) == 1
    assert call(stride=3) == 1 and call(beams=33, stride=33) == 2 and call(batch=1 << 16) == 2
    assert call(parent=FAKE + (1 << 24) + 2) == 3
    assert call(state=(None, 4, 64, 128, 1024)) == 1 and call(state=(FAKE, 0, 64, 128, 1024)) == 1
    assert call(state=(FAKE, 4, 64, 32, 1024)) == 1          # runs overlap
    assert call(state=(FAKE, 4, 64, 128, 256)) == 1          # beams overlap
    assert call(state=(FAKE, 1 << 31, 4, 4, 1 << 34), parent=1 << 45) == 2 and call(state=(FAKE, 1, 1 << 47, 0, 1 << 47)) == 2
    assert call(parent=FAKE + 64) == 1                        # parent inside the state
    assert call(count=2, more=[(FAKE, 1, 64, 0, 64)]) == 1   # the same state twice
    with pytest.raises(ValueError):
        q.make_beam_states([torch.zeros(4, 8)])
