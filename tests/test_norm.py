"""Residual addition and root-mean-square norm (bc_add_rmsnorm,
bc_add_rmsnorm_q8) against the formula in 64 bits, and the refusals."""
import numpy as np
import pytest
import torch

EPS = 1e-6
FAKE = 0x10000                    # aligned non-null address: never dereferenced
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _step(dtype):
    return torch.finfo(dtype).eps / 2


def _rel(D):
    """Relative error of the kernels' fp32 norm.  A thread adds t squares in a
    row (16 at most while a row fits a block, D / 1024 beyond), ten shuffle
    steps and one block sum follow: (t + 11) roundings of 2^-24 on the mean,
    half of that on its root; then the division, eps, the root, two products
    and h's own rounding (once in v, once in each square): 8 more."""
    t = max(16, (D + 1023) // 1024 + 8)
    return ((t + 11) / 2 + 8) * 2.0 ** -24


def _inputs(M, D, xt, rt, wt, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, D), generator=g).to(xt).cuda()
    r = (3 * torch.randn((M, D), generator=g)).to(rt).cuda() if rt else None
    w = (1 + 0.3 * torch.randn((D,), generator=g)).to(wt).cuda() if wt else None
    return x, r, w


def _formula(x, r, w):
    h = x.double() if r is None else x.double() + r.double()
    v = h / torch.sqrt((h * h).mean(dim=-1, keepdim=True) + EPS)
    return h, v if w is None else v * w.double()


def _near(got, want, rel, floor=0.0):
    err = (got.double() - want).abs()
    assert bool((err <= rel * want.abs() + floor).all()), float((err / (want.abs() + 1e-30)).max())


@pytest.mark.gpu
@pytest.mark.parametrize("xt,rt,wt,ot", [(F32, F32, F16, F32), (F32, BF16, BF16, BF16), (BF16, None, BF16, BF16),
                                         (F16, F16, F32, F16), (F32, None, None, F32), (BF16, F32, None, F16)])
@pytest.mark.parametrize("M,D", [(1, 1), (1, 896), (3, 7), (5, 63), (2, 64), (70, 128), (9, 200), (4, 257), (3, 512),
                                 (2, 1000), (2, 1001), (3, 1024), (2, 2048), (2, 4095), (2, 4096), (1, 8192),
                                 (1, 16384), (2, 16392), (1, 20001)])
def test_norm(cuda_lib, M, D, xt, rt, wt, ot):
    x, r, w = _inputs(M, D, xt, rt, wt, 1000 * M + D)
    h, v = _formula(x, r, w)
    x0 = x.clone()
    out = cuda_lib.add_rmsnorm(x, w, EPS, residual=r, out_dtype=ot)
    assert out.dtype == ot and torch.equal(x, x0)
    # one more rounding to the output's type (2^-25: half of fp16's least step)
    _near(out, v, _rel(D) + (_step(ot) if ot != F32 else 0), 2.0 ** -25)
    if r is not None:
        _near(r, h, 2.0 ** -24 + _step(r.dtype), 2.0 ** -25)


@pytest.mark.gpu
@pytest.mark.parametrize("xt,rt,wt,ot", [(F32, F32, F16, F32), (BF16, BF16, BF16, BF16), (F16, None, None, F32)])
@pytest.mark.parametrize("M,D", [(3001, 264), (2400, 704), (1500, 1344), (700, 4088)])
def test_norm_of_many_rows(cuda_lib, M, D, xt, rt, wt, ot):
    """Enough rows that a block takes several."""
    x, r, w = _inputs(M, D, xt, rt, wt, D)
    h, v = _formula(x, r, w)
    res = r if r is None else r.clone()
    _near(cuda_lib.add_rmsnorm(x, w, EPS, residual=res, out_dtype=ot), v, _rel(D) + (_step(ot) if ot != F32 else 0), 2.0 ** -25)
    if r is not None:
        _near(res, h, 2.0 ** -24 + _step(r.dtype), 2.0 ** -25)
    if xt == ot:
        cuda_lib.add_rmsnorm(x, w, EPS, residual=r, out=x)
        _near(x, v, _rel(D) + (_step(ot) if ot != F32 else 0), 2.0 ** -25)


@pytest.mark.gpu
def test_norm_q8_of_many_rows(cuda_lib):
    x, r, w = _inputs(1600, 1344, F32, BF16, F16, 9)
    _, v = _formula(x, r, w)
    _check_q8(cuda_lib.add_rmsnorm_q8(x, w, EPS, residual=r), v, _rel(1344))


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 1, 2, 4])
def test_norm_of_unaligned_views(cuda_lib, shift):
    """Addresses that only have their element's alignment."""
    M, D = 3, 264
    buf = torch.randn(M * D + 8, device="cuda").to(BF16)
    x = buf[shift:shift + M * D].view(M, D)
    w = torch.randn(D + 1, device="cuda")[1:]
    _, v = _formula(x, None, w)
    out = torch.zeros(M * D + 8, device="cuda")
    got = cuda_lib.add_rmsnorm(x, w, EPS, out=out[shift:shift + M * D].view(M, D))
    _near(got, v, _rel(D))
    rest = torch.cat([out[:shift], out[shift + M * D:]])
    assert bool((rest == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [96, 1003, 4096, 17000])
def test_norm_in_place(cuda_lib, D):
    x, r, w = _inputs(4, D, F32, F32, F32, D)
    h, v = _formula(x, r, w)
    cuda_lib.add_rmsnorm(x, w, EPS, residual=r, out=x)
    _near(x, v, _rel(D))
    _near(r, h, 2.0 ** -23)


@pytest.mark.gpu
def test_norm_of_zero_and_spread_rows(cuda_lib):
    x = torch.zeros((4, 640), device="cuda")
    x[1] = 1e-15
    x[2, 5] = 1e15                                   # its square is far below fp32's largest
    x[3] = torch.logspace(-18, 12, 640, device="cuda")
    _, v = _formula(x, None, None)
    out = cuda_lib.add_rmsnorm(x, None, EPS)
    assert bool((out[0] == 0).all())
    _near(out, v, _rel(640), 1e-37)


@pytest.mark.gpu
@pytest.mark.parametrize("xt,rt,wt", [(F32, F32, F16), (BF16, BF16, BF16), (F16, None, F32)])
@pytest.mark.parametrize("M,D", [(1, 64), (3, 128), (5, 896), (2, 4096), (1, 4864), (2, 16384), (1, 16448)])
def test_norm_q8(cuda_lib, M, D, xt, rt, wt):
    x, r, w = _inputs(M, D, xt, rt, wt, D + M)
    h, v = _formula(x, r, w)
    _check_q8(cuda_lib.add_rmsnorm_q8(x, w, EPS, residual=r), v, _rel(D))
    if r is not None:
        _near(r, h, 2.0 ** -24 + _step(r.dtype))


def _check_q8(out, v, rel):
    codes, s, z = out
    v = v.view(v.shape[0], -1, 64)
    q, s, z = codes.view(v.shape).double(), s.double(), z.double()
    lo, hi = v.amin(-1).clamp(max=0), v.amax(-1).clamp(min=0)
    want = ((hi - lo) / 255).clamp(min=2.0 ** -24, max=65504)
    # one rounding to fp16 (2^-25: half its least step) of a value a few fp32 roundings off
    _near(s, want, 2.0 ** -11 * 1.001 + 2 * rel, 2.0 ** -25)
    # zero and codes are those of the stored scale; a quotient may be `off` beside its border
    off = 255 * (2 * rel + 2.0 ** -23)
    assert bool(((z - (-lo / s).clamp(max=255)).abs() <= 0.5 + off).all())
    ideal = v / s[..., None]
    low, high = -z[..., None], 255 - z[..., None]
    assert bool(((q - z[..., None] - torch.minimum(torch.maximum(ideal, low), high)).abs() <= 0.5 + off).all())


@pytest.mark.gpu
def test_norm_q8_edges(cuda_lib):
    """Groups of zeros, of one sign, of one value, and with an outlier."""
    x = torch.zeros((1, 384), device="cuda")
    x[0, 64:128] = 0.5
    x[0, 128:192] = -torch.rand(64, device="cuda") - 0.1
    x[0, 192:256] = 1e-6 * torch.randn(64, device="cuda")
    x[0, 256] = 100
    x[0, 320:384] = torch.linspace(-3, 3, 64, device="cuda")
    _, v = _formula(x, None, None)
    out = cuda_lib.add_rmsnorm_q8(x, None, EPS)
    _check_q8(out, v, _rel(384))
    assert bool((out[0][0, :64] == 0).all()) and float(out[2][0, 0]) == 0
    assert float(out[2][0, 1]) == 0 and float(out[2][0, 2]) == 255


@pytest.mark.gpu
def test_q8_rows_are_packed_weights(cuda_lib):
    """The 8-bit form read back by matmul_q (packed, 8 bits) with unit rows."""
    D = 128
    x, _, w = _inputs(6, D, F32, None, F16, 5)
    codes, s, z = cuda_lib.add_rmsnorm_q8(x, w, EPS)
    eye = torch.eye(D, device="cuda")
    y = cuda_lib.matmul_q(eye, codes, s, z, 8, 64, cuda_lib.BC_MODE_PACKED)       # [D][6]
    want = (codes.view(6, -1, 64).double() - z.double()[..., None]) * s.double()[..., None]
    _near(y.T, want.view(6, D), 1e-4)


def test_norm_rejects_on_host():
    import quantized_matmul_02_b200 as q
    f = q.lib.bc_add_rmsnorm
    ok = [FAKE, 0, FAKE + (1 << 20), 0, FAKE + (2 << 20), 0, 4, 64, EPS, FAKE + (3 << 20), 0, None]

    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    assert call(_0=None) == 1 and call(_9=None) == 1
    assert call(_6=0) == 1 and call(_7=0) == 1 and call(_7=-1) == 1 and call(_6=1 << 25) == 2
    assert call(_8=0.0) == 1 and call(_8=float("nan")) == 1 and call(_8=float("inf")) == 1
    assert call(_1=5) == 2 and call(_3=9) == 2 and call(_5=-1) == 2 and call(_10=7) == 2
    assert call(_0=FAKE + 2) == 3 and call(_2=FAKE + 1) == 3
    assert call(_9=FAKE, _10=1) == 1                 # out over x, another type
    assert call(_9=FAKE + 64) == 1                   # out into x
    assert call(_2=FAKE) == 1                        # residual over x
    assert call(_9=FAKE + (2 << 20)) == 1            # out over the weight
    g = q.lib.bc_add_rmsnorm_q8
    a = [FAKE, 0, None, 0, None, 0, 4, 64, EPS, FAKE + (1 << 20), FAKE + (2 << 20), FAKE + (3 << 20), None]
    assert g(*a[:7], 65, *a[8:]) == 1 and g(*a[:10], None, *a[11:]) == 1
    assert g(*a[:9], FAKE + (1 << 20) + 4, *a[10:]) == 3
    assert g(*a[:11], FAKE + (2 << 20), None) == 1   # zeros over the scales
    with pytest.raises(ValueError):
        q.add_rmsnorm(torch.zeros(2, 8), None)       # not on a GPU


@pytest.mark.gpu
def test_norm_wrapper_refuses(cuda_lib):
    x = torch.zeros((2, 64), device="cuda")
    for bad in (dict(residual=x[:1].clone()), dict(out=torch.empty((2, 63), device="cuda")),
                dict(out_dtype=torch.int32), dict(residual=torch.zeros((2, 128), device="cuda")[:, ::2])):
        with pytest.raises(ValueError):
            cuda_lib.add_rmsnorm(x, None, **bad)
    with pytest.raises(ValueError):
        cuda_lib.add_rmsnorm_q8(x[:, :32].contiguous(), None)
    with pytest.raises(cuda_lib.BCError):
        cuda_lib.add_rmsnorm(x, None, eps=-1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("M,D", [(2, 96), (2, 256), (3, 257), (2, 320), (1, 896), (3, 1003), (2, 4096), (2, 16392), (1, 20001),
                                 (3001, 1344)])
def test_norm_of_the_largest_values(cuda_lib, M, D):
    """Values up to 1e18: the sum of their squares is beyond fp32 from 341 on."""
    g = torch.Generator().manual_seed(D)
    x = torch.rand((M, D), generator=g) * 2 - 1
    if M > 1:
        x[1] = torch.sign(x[1])
    x = (x * 1e18).cuda()
    _, v = _formula(x, None, None)
    _near(cuda_lib.add_rmsnorm(x, None, EPS), v, _rel(D))
    if D % 64 == 0:
        _check_q8(cuda_lib.add_rmsnorm_q8(x, None, EPS), v, _rel(D))


def _rows_that_stream(D):
    """From here on a block stays and takes rows in turn: four rows for each of
    the blocks of D / 8 threads (in warps) that 148 SMs hold, 1024 threads each."""
    return 4 * 148 * (1024 // ((D // 8 + 31) // 32 * 32))


@pytest.mark.gpu
@pytest.mark.parametrize("xt,rt,wt,ot", [(F32, F32, F16, F32), (BF16, BF16, BF16, BF16), (F16, None, None, F32)])
@pytest.mark.parametrize("D", [264, 320, 520, 704, 1024, 1032, 1536, 2048, 2056, 2560, 4088])
@pytest.mark.parametrize("more", [0, 1, 997])
def test_norm_of_rows_in_turn(cuda_lib, D, more, xt, rt, wt, ot):
    """Each width of block, with a full and a partly filled last warp."""
    M = _rows_that_stream(D) + more
    x, r, w = _inputs(M, D, xt, rt, wt, D)
    h, v = _formula(x, r, w)
    res = r if r is None else r.clone()
    last = _step(ot) if ot != F32 else 0
    _near(cuda_lib.add_rmsnorm(x, w, EPS, residual=res, out_dtype=ot), v, _rel(D) + last, 2.0 ** -25)
    if r is not None:
        _near(res, h, 2.0 ** -24 + _step(r.dtype), 2.0 ** -25)
    if xt == ot:
        cuda_lib.add_rmsnorm(x, w, EPS, residual=r, out=x)
        _near(x, v, _rel(D) + last, 2.0 ** -25)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [320, 576, 960, 1088, 1984, 2112, 4032])
def test_norm_q8_of_rows_in_turn(cuda_lib, D):
    x, r, w = _inputs(_rows_that_stream(D) + 3, D, F32, BF16, F16, D)
    h, v = _formula(x, r, w)
    _check_q8(cuda_lib.add_rmsnorm_q8(x, w, EPS, residual=r), v, _rel(D))
    _near(r, h, 2.0 ** -24 + _step(BF16), 2.0 ** -25)
