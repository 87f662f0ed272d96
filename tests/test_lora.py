"""Low-rank adapters of many requests (bc_lora_add, bc_lora_add_batched)
against the formula in 64 bits, and the refusals."""
import ctypes
import math
import weakref

import pytest
import torch

FAKE = 0x10000                    # aligned non-null address: never dereferenced
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _make(M, K, Ns, R, n, xt, wt, seed, mixed=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = r(M, K).to(xt)
    mats = [((r(n, R, K) / math.sqrt(K)).to(wt), (r(n, N, R) / math.sqrt(R)).to(wt), r(M, N)) for N in Ns]
    ranks = torch.randint(0, R + 1, (n,), generator=g, device="cuda", dtype=torch.int32) if mixed else None
    scaling = 0.2 + torch.rand((n,), generator=g, device="cuda")
    return x, mats, ranks, scaling


def _check(x, A, B, y0, y, start, adapter, ranks, scaling):
    """Every row against the formula; rows without an adapter unchanged.

    Bound, relative to S = |c| sum_r (sum_k |A x|) |B|: an fp32 x enters as two
    tf32 pieces, v as pieces of B's type, each at most 2^-22 away; a tensor-core
    step of k products is taken as k + 1 additions of 2^-23.  Eight warps share
    K at least, so a warp has at most ceil(K / 256) pieces of 32, each of 8 steps
    of 8 (or fewer additions: 2 of 16) and at most one addition to join it; up
    to 8 + 8 additions join the warps and the parts of K, and the scale is one
    product.  16 ranks take at most 3 steps of 16.  Then y: one addition (2^-24
    of the result)."""
    n, R, K = A.shape
    rel = 2 * 2.0 ** -22 + ((8 * 9 + 1) * math.ceil(K / 256) + 17 + 3 * 17 * math.ceil(R / 16)) * 2.0 ** -23
    seen = torch.zeros(x.shape[0], dtype=torch.bool)
    for i in range(len(adapter)):
        a, s0, s1 = int(adapter[i]), int(start[i]), int(start[i + 1])
        keep = 0 if a < 0 or a >= n else R if ranks is None else int(ranks[a])
        if keep == 0 or s0 == s1:
            continue
        seen[s0:s1] = True
        c = 1.0 if scaling is None else float(scaling[a])
        Ad, Bd, xd = A[a, :keep].double(), B[a, :, :keep].double(), x[s0:s1].double()
        want = y0[s0:s1].double() + c * (xd @ Ad.T) @ Bd.T
        S = abs(c) * (xd.abs() @ Ad.abs().T) @ Bd.abs().T
        err = (y[s0:s1].double() - want).abs()
        bound = rel * S + 2.0 ** -24 * (want.abs() + rel * S)
        assert bool((err <= bound).all()), (i, a, float((err / bound).max()))
    assert torch.equal(y[~seen], y0[~seen])


def _run(q, x, mats, start, adapter, ranks, scaling):
    st = torch.tensor(start, dtype=torch.int32, device="cuda")
    ad = torch.tensor(adapter, dtype=torch.int32, device="cuda")
    old = [m[2].clone() for m in mats]
    q.lora_add_batched(q.make_lora_descs([(x, A, B, y) for A, B, y in mats]), st, ad, ranks, scaling)
    for (A, B, y), y0 in zip(mats, old):
        _check(x, A, B, y0, y, start, adapter, ranks, scaling)


@pytest.mark.gpu
@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("wt", [F16, BF16])
@pytest.mark.parametrize("M,K,Ns,R,n", [
    (1, 64, (1,), 8, 1), (1, 896, (896, 128, 128), 16, 4), (3, 128, (33,), 8, 2), (17, 192, (100, 64), 24, 3),
    (64, 1024, (260,), 32, 20), (130, 320, (77,), 64, 40), (256, 448, (129,), 128, 7), (256, 64, (32,), 16, 1)])
def test_decode_one_row_a_request(cuda_lib, M, K, Ns, R, n, xt, wt):
    x, mats, ranks, scaling = _make(M, K, Ns, R, n, xt, wt, M + K)
    g = torch.Generator().manual_seed(M)
    adapter = torch.randint(-1, n + 1, (M,), generator=g).tolist()    # some without one, on both sides
    if M == 1:
        adapter = [n - 1]
        ranks = None
    _run(cuda_lib, x, mats, list(range(M + 1)), adapter, ranks, scaling)


@pytest.mark.gpu
@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("wt", [F16, BF16])
@pytest.mark.parametrize("start,K,Ns,R", [
    ([0, 300], 128, (64,), 16), ([0, 1, 2, 259], 192, (36, 31), 8), ([0, 0, 100, 100, 257, 400], 896, (130,), 32),
    ([5, 70, 200, 390], 256, (40,), 128), ([0, 64, 128, 192, 256, 320], 64, (256,), 40),
    ([0, 1000], 2176, (45,), 24), ([0, 3, 17, 33, 66, 130, 259, 516, 1030], 128, (68,), 16)])
def test_prompts(cuda_lib, start, K, Ns, R, xt, wt):
    S, M = len(start) - 1, start[-1] + 10                             # rows behind the last segment
    x, mats, ranks, scaling = _make(M, K, Ns, R, 3, xt, wt, M + K)
    if ranks is not None:
        ranks[0] = R
    _run(cuda_lib, x, mats, start, [i % 4 - (i == 5) for i in range(S)], ranks, scaling)


@pytest.mark.gpu
def test_many_short_segments(cuda_lib):
    """More rows than are ordered by adapter, in segments of 0 to 5 rows."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 6, (700,), generator=g).tolist()
    start = [0]
    for n in lens:
        start.append(start[-1] + n)
    x, mats, ranks, scaling = _make(start[-1], 128, (50,), 16, 9, F32, BF16, 4)
    _run(cuda_lib, x, mats, start, torch.randint(-1, 9, (700,), generator=g).tolist(), ranks, scaling)


@pytest.mark.gpu
def test_no_rows_no_ranks(cuda_lib):
    """Segments that are all empty, all without an adapter, or of rank 0."""
    x, mats, _, scaling = _make(40, 64, (24,), 8, 2, F32, F16, 5)
    y0 = mats[0][2].clone()
    for start, adapter, ranks in (([0, 0, 0], [0, 1], None), ([0, 20, 40], [-1, 2], None), ([0, 20, 40], [0, 1], [0, -3])):
        rk = None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device="cuda")
        _run(cuda_lib, x, mats, start, adapter, rk if rk is None else rk.clamp(min=0), scaling)
        assert torch.equal(mats[0][2], y0)


@pytest.mark.gpu
def test_unused_ranks_and_rows_are_not_read(cuda_lib):
    """NaN behind an adapter's rank, in other adapters and in rows of no
    segment stays out of the results; places outside 0..M are cut."""
    M, K, N, R = 24, 128, 40, 16
    for rank in (1, 5, 8, 13):
        x, mats, _, scaling = _make(M, K, (N,), R, 3, F32, BF16, rank)
        A, B, y = mats[0]
        ranks = torch.full((3,), rank, dtype=torch.int32, device="cuda")
        A[:, rank:] = float("nan")
        B[:, :, rank:] = float("nan")
        A[2], B[2] = float("nan"), float("nan")
        x[20:] = float("nan")
        _run(cuda_lib, x, mats, [0, 9, 20], [1, 0], ranks, scaling)
        assert not torch.isnan(y).any()
    x, mats, ranks, scaling = _make(M, K, (N,), R, 3, F32, F16, 9, mixed=False)
    y0 = mats[0][2].clone()
    st = torch.tensor([-5, 10, 1000], dtype=torch.int32, device="cuda")
    ad = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    cuda_lib.lora_add(x, mats[0][0], mats[0][1], mats[0][2], st, ad, scaling=scaling)
    _check(x, *mats[0][:2], y0, mats[0][2], [0, 10, M], [1, 0], None, scaling)


@pytest.mark.gpu
def test_same_bits_every_time_and_unaligned_y(cuda_lib):
    x, mats, ranks, scaling = _make(300, 512, (96,), 32, 4, BF16, BF16, 11)
    A, B, y = mats[0]
    start = torch.tensor([0, 100, 101, 300], dtype=torch.int32, device="cuda")
    adapter = torch.tensor([0, 3, 2], dtype=torch.int32, device="cuda")
    buf = torch.zeros(300 * 96 + 1, device="cuda")
    off = buf[1:].view(300, 96)                       # rows that begin off 16 bytes
    off.copy_(y)
    y2 = y.clone()
    for t in (y, y2, off):
        cuda_lib.lora_add(x, A, B, t, start, adapter, ranks, scaling)
    assert torch.equal(y, y2) and torch.equal(y, off)


@pytest.mark.gpu
def test_more_projections_than_one_launch(cuda_lib):
    x, mats, ranks, scaling = _make(5, 64, (16,) * 35, 8, 2, F32, F16, 12)
    _run(cuda_lib, x, mats, [0, 2, 5], [1, 0], None, None)


def test_lora_rejects_on_host():
    import quantized_matmul_02_b200 as q
    at = [FAKE + (i << 26) for i in range(8)]
    ok = dict(x=at[0], xt=0, A=at[1], B=at[2], wt=1, M=4, N=32, K=64, R=8, n=2, start=at[3], adapter=at[4], S=4,
              ranks=None, scaling=None, y=at[5], ws=at[6], wsb=1 << 20, stream=None)
    call = lambda **kw: q.lib.bc_lora_add(*{**ok, **kw}.values())  # noqa: E731
    for k in ("x", "A", "B", "start", "adapter", "y"):
        assert call(**{k: None}) == 1
    for k in ("M", "N", "K", "R", "n", "S"):
        assert call(**{k: 0}) == 1 and call(**{k: -8}) == 1
    assert call(K=96) == 1 and call(R=12) == 1 and call(R=136) == 2 and call(S=4097) == 2
    assert call(xt=1) == 2 and call(wt=0) == 2 and call(M=1 << 25) == 2 and call(N=1 << 30) == 2
    assert call(x=at[0] + 8) == 3 and call(A=at[1] + 2) == 3 and call(y=at[5] + 2) == 3 and call(start=at[3] + 1) == 3
    assert call(ws=None) == 4 and call(wsb=64) == 4 and call(ws=at[6] + 8) == 3 and call(ws=at[5]) == 1
    assert call(y=at[0]) == 1 and call(y=at[2] + 64) == 1 and call(y=at[3]) == 1
    arr = (q.LoraDesc * 2)(*[q.LoraDesc(at[0], at[1], at[2], at[5], 32, 64)] * 2)
    assert q.lib.bc_lora_add_batched(arr, 2, 4, 8, 2, 0, 1, at[3], at[4], 4, None, None, at[6], 1 << 20, None) == 1   # one y twice
    assert q.lib.bc_lora_add_batched(None, 1, 4, 8, 2, 0, 1, at[3], at[4], 4, None, None, at[6], 1 << 20, None) == 1
    with pytest.raises(ValueError):
        q.make_lora_descs([(torch.zeros(2, 64), torch.zeros(1, 8, 64).half(), torch.zeros(1, 4, 8).half(), torch.zeros(2, 4))])
    with pytest.raises(ValueError):
        q.make_lora_descs([])


@pytest.mark.gpu
def test_lora_wrapper_refuses(cuda_lib):
    x, mats, _, scaling = _make(4, 64, (24,), 8, 2, F32, F16, 5)
    A, B, y = mats[0]
    st = torch.arange(5, dtype=torch.int32, device="cuda")
    ad = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in ((x, A, B[:, :20].contiguous(), y, st, ad), (x, A, B, y[:3], st, ad), (x, A, B.float(), y, st, ad),
                (x, A, B, y, st[:4], ad), (x, A, B, y, st.long(), ad), (x.half(), A, B, y, st, ad),
                (x, A, B, y.cpu(), st, ad), (x, A.transpose(1, 2), B, y, st, ad)):
        with pytest.raises(ValueError):
            cuda_lib.lora_add(*bad)


class _OnGpu:
    """What the wrappers ask of a CUDA tensor, without one."""

    def __init__(self, shape, dtype):
        self._t = torch.empty(shape, dtype=dtype)
        self.shape, self.dtype = self._t.shape, dtype
        self.dim, self.stride, self.numel = self._t.dim, self._t.stride, self._t.numel
        self.is_contiguous, self.data_ptr, self.element_size = self._t.is_contiguous, self._t.data_ptr, self._t.element_size

    def get_device(self):
        return 0


def test_descriptors_hold_their_tensors():
    """A list that is cleared or refilled after the call takes nothing away."""
    import quantized_matmul_02_b200 as q
    made = lambda: [_OnGpu((4, 64), F32), _OnGpu((2, 8, 64), F16), _OnGpu((2, 24, 8), F16), _OnGpu((4, 24), F32)]  # noqa: E731
    items = [made(), made()]
    alive = [weakref.ref(t) for i in items for t in i]
    d = q.make_lora_descs(items)
    items[0].clear()
    items.clear()
    assert all(r() is not None for r in alive) and d.count == 2
    del d
    assert all(r() is None for r in alive)
    states = [_OnGpu((4, 8), F32), _OnGpu((4, 3, 8), BF16)]
    alive = [weakref.ref(t) for t in states]
    st = q.make_beam_states(states)
    states.clear()
    assert all(r() is not None for r in alive) and st.count == 2


@pytest.mark.parametrize("where", range(7))
def test_lora_refuses_scratch_over_what_it_reads(where):
    """x, A, B, the segments, the adapters, ranks and scaling: from their first
    byte, and scratch that only reaches their first."""
    import quantized_matmul_02_b200 as q
    at = [FAKE + (i << 26) for i in range(10)]
    M, N, K, R, n, S = 4, 32, 64, 8, 2, 4
    d = q.LoraDesc(at[0], at[1], at[2], at[3], N, K)
    need = q.lib.bc_workspace_size_lora(ctypes.byref(d), 1, M, R, n, S, 0)
    target = (at[0], at[1], at[2], at[4], at[5], at[6], at[7])[where]
    for ws in (target, target - (need - 1) // 256 * 256):
        assert q.lib.bc_lora_add(at[0], 0, at[1], at[2], 1, M, N, K, R, n, at[4], at[5], S, at[6], at[7], at[3],
                                 ws, need, None) == 1


def _exact(x, A, B, start, adapter, ranks, scaling):
    """c B (A x) of each row in 64 bits."""
    out = torch.zeros((x.shape[0], B.shape[1]), dtype=torch.float64, device=x.device)
    for i, a in enumerate(adapter):
        keep = A.shape[1] if ranks is None else int(ranks[a])
        s = slice(start[i], start[i + 1])
        out[s] = float(scaling[a]) * (x[s].double() @ A[a, :keep].double().T) @ B[a, :, :keep].double().T
    return out


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("wt", [F16, BF16])
@pytest.mark.parametrize("start,K,N,R", [
    (list(range(65)), 2176, 260, 32), (list(range(0, 65, 8)), 896, 130, 128), (list(range(41)), 4096, 130, 16),
    ([0, 300, 777], 4864, 896, 128), ([0, 100, 400], 2176, 100, 24), ([0, 1000], 1024, 333, 64)])
def test_every_piece_counts(cuda_lib, start, K, N, R, xt, wt):
    """The root of the mean squared error over random signs, relative to that of
    the result, where the worst case of every rounding at once says little.
    Expected: an fp32 x in two tf32 pieces and v in pieces, at most 2^-22 of a
    value off and below 2^-23 in this mean, each; sums in parts of 16 tensor-core
    steps that lose up to an accumulator's last bit, 2^-23 of what they hold, on
    average half of it, and no part larger than the whole: sqrt(16) * 2^-24 =
    2^-22 if they were independent, for A x, and (3 * R / 16)^0.5 * 2^-24 for B v,
    2^-21.7 at rank 128; roots of squares: 2^-21.  Losses of one part have one sign,
    so twice that is allowed, 2^-20.  One piece less is far above: x in one tf32
    piece 2^-13, v in two bf16 pieces 2^-18, v in one fp16 piece 2^-13."""
    n, M = 5, start[-1]
    x, mats, _, scaling = _make(M, K, (N,), R, n, xt, wt, K + N, mixed=False)
    A, B, _ = mats[0]
    adapter = [i % n for i in range(len(start) - 1)]
    y = torch.zeros((M, N), device="cuda")
    cuda_lib.lora_add(x, A, B, y, _ints(start), _ints(adapter), scaling=scaling)
    want = _exact(x, A, B, start, adapter, None, scaling)
    rel = float((y.double() - want).norm() / want.norm())
    assert rel <= 2.0 ** -20, rel * 2 ** 24


@pytest.mark.gpu
@pytest.mark.parametrize("xt,M", [(F32, 4900), (BF16, 9600)])
@pytest.mark.parametrize("wt", [F16, BF16])
@pytest.mark.parametrize("K", [4096, 12288])
def test_long_sums_are_taken_in_parts(cuda_lib, K, M, xt, wt):
    """Enough rows that K is not divided among blocks, and values of one sign, so
    that what the tensor cores cut off adds up.  A step cuts off half of the
    accumulator's last bit on average, up to 2^-24 of it: a part of 16 steps
    loses 16 * 2^-24 / 2 = 2^-21 of itself, as its sum grows; v's three steps and
    the other roundings are beside it.  In one sum K = 12288 takes 96 steps a warp
    or more, which would lose 2^-18.4."""
    R, N = 16, 24
    g = torch.Generator(device="cuda").manual_seed(K)
    x = (0.5 + torch.rand((M, K), generator=g, device="cuda")).to(xt)
    A = ((0.5 + torch.rand((2, R, K), generator=g, device="cuda")) / K).to(wt)
    B = (0.5 + torch.rand((2, N, R), generator=g, device="cuda")).to(wt)
    y, scaling = torch.zeros((M, N), device="cuda"), torch.ones(2, device="cuda")
    start, adapter = [0, M // 3, M], [1, 0]
    cuda_lib.lora_add(x, A, B, y, _ints(start), _ints(adapter), scaling=scaling)
    want = _exact(x, A, B, start, adapter, None, scaling)
    lost = float(((want - y.double()) / want).mean())
    assert abs(lost) <= 2.0 ** -20, lost * 2 ** 24
    x2, mats, ranks, scaling = _make(M, K, (N,), R, 3, xt, wt, K, mixed=False)
    A, B, y = mats[0][0], mats[0][1], torch.zeros((M, N), device="cuda")
    cuda_lib.lora_add(x2, A, B, y, _ints(start), _ints(adapter), scaling=scaling)
    want = _exact(x2, A, B, start, adapter, None, scaling)
    assert float((y.double() - want).norm() / want.norm()) <= 2.0 ** -20
