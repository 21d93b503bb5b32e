"""Layer normalisation on the GPU against the 64-bit definition, with bounds
derived from the operations (tests/operator_reference.py)."""

import pytest
import torch

from tests import operator_reference as ref

pytestmark = pytest.mark.gpu

DT = ref.DTYPES


def rows_of(seed, rows, width, dtype, shift=0.25):
    gen = torch.Generator().manual_seed(seed)
    scale = torch.exp(0.5 * torch.randn(width, generator=gen, dtype=torch.float64))
    return (torch.randn(rows, width, generator=gen, dtype=torch.float64) * scale + shift).to(dtype)


def within(got, want, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, what
    off = (got - want).abs()
    assert bool((off <= bound).all()), f"{what}: worst error/bound {float((off / bound).max()):.3g}"


def run_forward(tg, x, w, b, eps=1e-5, **kw):
    dev = [t.cuda() if t is not None else None for t in (x, w, b)]
    return tg.layer_norm(*dev, eps, stats=True, **kw)


def check_forward(x, w, b, out, eps=1e-5):
    y, mean, rstd = out
    ry, rm, rr = ref.layer_norm(x, w, b, eps)
    c = ref.chain(x.shape[-1])
    within(y, ry, ref.layer_norm_bound(x, w, b, eps), "y")
    within(mean, rm, c * x.double().abs().mean(-1) + ref.tiny(torch.float32), "mean")
    spread = x.double().abs().mean(-1)
    within(rstd, rr, rr * (c + 6 * ref.U) + rr ** 3 * (c * spread) ** 2, "rstd")


def check_backward(tg, x, dy, w, stride_pad=0):
    _, mean, rstd = (t for t in ref.layer_norm(x, None, None, 1e-5))
    mean, rstd = mean.float(), rstd.float()
    dev = [t.cuda() if t is not None else None for t in (dy, x, mean, rstd, w)]
    if stride_pad:
        for i in (0, 1):
            wide = torch.full((x.shape[0], x.shape[1] + stride_pad), float("nan"), dtype=x.dtype, device="cuda")
            wide[:, :x.shape[1]] = dev[i]
            dev[i] = wide[:, :x.shape[1]]
    got = tg.layer_norm_backward(*dev)
    want = ref.layer_norm_backward(dy, x, mean, rstd, w)
    bounds = ref.layer_norm_backward_bounds(dy, x, mean, rstd, w)
    for name, g, r, b in zip(("dx", "dweight", "dbias"), got, want, bounds):
        within(g, r, b, name)
    return got


WIDTHS = [1, 2, 7, 8, 31, 64, 100, 512, 520, 1000, 1024, 1028, 3001, 4096, 4104, 8200, 16384, 17000, 70000]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("width", WIDTHS)
def test_forward_and_backward_widths(cuda_lib, width, dtype):
    dt = DT[dtype]
    rows = 3 if width > 16384 else 37
    x, dy = rows_of(1, rows, width, dt), rows_of(2, rows, width, dt, shift=0.0)
    w, b = rows_of(3, 1, width, dt, shift=1.0)[0], rows_of(4, 1, width, dt)[0]
    check_forward(x, w, b, run_forward(cuda_lib, x, w, b))
    check_backward(cuda_lib, x, dy, w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 2, 5, 151, 153, 2500])
@pytest.mark.parametrize("width", [24, 333, 1280])
def test_row_counts_with_single_precision_weights(cuda_lib, rows, width, dtype):
    dt = DT[dtype]
    x, dy = rows_of(5, rows, width, dt), rows_of(6, rows, width, dt, shift=0.0)
    w, b = rows_of(7, 1, width, torch.float32, shift=1.0)[0], rows_of(8, 1, width, torch.float32)[0]
    check_forward(x, w, b, run_forward(cuda_lib, x, w, b))
    dw = check_backward(cuda_lib, x, dy, w)[1]
    assert dw.dtype == torch.float32


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,width", [(12000, 61), (6000, 257), (5000, 1001), (3000, 2047), (700, 8185), (4000, 4099)])
def test_many_rows_that_start_on_no_boundary(cuda_lib, rows, width, dtype):
    """Every shift from the 16-byte boundary, several rows per group, and each kind of weight."""
    dt = DT[dtype]
    x, dy = rows_of(31, rows, width, dt), rows_of(32, rows, width, dt, shift=0.0)
    w, b = rows_of(33, 1, width, dt, shift=1.0)[0], rows_of(34, 1, width, dt)[0]
    check_forward(x, w, b, run_forward(cuda_lib, x, w, b))
    check_backward(cuda_lib, x, dy, w)


@pytest.mark.parametrize("dtype,weights", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("rows,width", [(200, 8200), (310, 11111), (480, 16384), (160, 16370)])
def test_many_wide_rows(cuda_lib, rows, width, dtype, weights):
    """Rows whose weights do not fit the registers, several for a CTA."""
    dt, wt = DT[dtype], DT[weights]
    x, dy = rows_of(41, rows, width, dt), rows_of(42, rows, width, dt, shift=0.0)
    w, b = rows_of(43, 1, width, wt, shift=1.0)[0], rows_of(44, 1, width, wt)[0]
    check_forward(x, w, b, run_forward(cuda_lib, x, w, b))
    check_forward(x, w, None, run_forward(cuda_lib, x, w, None))
    check_forward(x, None, b, run_forward(cuda_lib, x, None, b))
    check_backward(cuda_lib, x, dy, w)
    check_backward(cuda_lib, x, dy, None)


@pytest.mark.parametrize("have_w,have_b", [(False, False), (True, False), (False, True)])
def test_weight_and_bias_are_optional(cuda_lib, have_w, have_b):
    x, dy = rows_of(9, 20, 264, torch.float16), rows_of(10, 20, 264, torch.float16)
    w = rows_of(11, 1, 264, torch.float16, shift=1.0)[0] if have_w else None
    b = rows_of(12, 1, 264, torch.float16)[0] if have_b else None
    check_forward(x, w, b, run_forward(cuda_lib, x, w, b))
    check_backward(cuda_lib, x, dy, w)


@pytest.mark.parametrize("pad,offset", [(8, 0), (5, 0), (3, 1), (8, 8)])
def test_strided_and_misaligned_rows(cuda_lib, pad, offset):
    """Rows apart from one another, starting on and off the vector boundary; what lies between stays out."""
    tg, width = cuda_lib, 512
    x = rows_of(13, 11, width, torch.bfloat16)
    wide = torch.full((11, width + pad + offset), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = wide[:, offset:offset + width]
    view.copy_(x.cuda())
    w = rows_of(14, 1, width, torch.bfloat16, shift=1.0)[0]
    y, mean, rstd = tg.layer_norm(view, w.cuda(), None, stats=True)
    assert y.is_contiguous()
    check_forward(x, w, None, (y, mean, rstd))
    check_backward(tg, x, rows_of(15, 11, width, torch.bfloat16), w, stride_pad=pad)


def test_leading_dimensions_and_no_rows(cuda_lib):
    tg = cuda_lib
    x = rows_of(16, 24, 40, torch.float32)
    y, mean, rstd = tg.layer_norm(x.view(2, 3, 4, 40).cuda(), stats=True)
    assert y.shape == (2, 3, 4, 40) and mean.shape == (24,)
    check_forward(x, None, None, (y.reshape(24, 40), mean, rstd))
    e = torch.empty((0, 40), device="cuda")
    assert tg.layer_norm(e).shape == (0, 40)
    s = torch.empty(0, device="cuda")
    dx, dw, db = tg.layer_norm_backward(e, e, s, s)
    assert dx.shape == (0, 40) and not dw.any() and not db.any()


def test_large_offset_and_constant_rows(cuda_lib):
    """The variance of rows far from zero comes from differences, not from a difference of sums of squares."""
    x = rows_of(17, 9, 2048, torch.float32, shift=1000.0)
    x[4] = 3.5
    check_forward(x, None, None, run_forward(cuda_lib, x, None, None))


def test_nan_and_infinity_stay_in_their_row(cuda_lib):
    tg = cuda_lib
    x = rows_of(18, 64, 768, torch.float16)
    clean = tg.layer_norm(x.cuda())
    x[7, 5], x[20, 700], x[40, 0] = float("nan"), float("inf"), float("-inf")
    y = tg.layer_norm(x.cuda())
    bad = torch.zeros(64, dtype=torch.bool)
    bad[[7, 20, 40]] = True
    assert torch.equal(y.isnan().any(1).cpu(), bad)
    assert torch.equal(y[~bad.cuda()], clean[~bad.cuda()])


def test_gradient_against_differences(cuda_lib):
    """The kernel's dx and dweight along random directions against central differences of the 64-bit forward pass."""
    rows, width, eps, h = 6, 129, 1e-5, 1e-5
    x, dy = rows_of(19, rows, width, torch.float32), rows_of(20, rows, width, torch.float32, shift=0.0)
    w, b = rows_of(21, 1, width, torch.float32, shift=1.0)[0], rows_of(22, 1, width, torch.float32)[0]
    _, mean, rstd = run_forward(cuda_lib, x, w, b, eps)
    dx, dw, db = (t.cpu().double() for t in cuda_lib.layer_norm_backward(dy.cuda(), x.cuda(), mean, rstd, w.cuda()))
    bounds = ref.layer_norm_backward_bounds(dy, x, mean.cpu(), rstd.cpu(), w)

    def loss(x, w, b):
        return float((dy.double() * ref.layer_norm(x, w, b, eps)[0]).sum())

    for i in range(3):
        v, vw, vb = (rows_of(30 + i, *shape, torch.float64) for shape in ((rows, width), (1, width), (1, width)))
        vw, vb = vw[0], vb[0]
        args = [x.double(), w.double(), b.double()]
        for k, (grad, dirn) in enumerate(((dx, v), (dw, vw), (db, vb))):
            up, down = list(args), list(args)
            up[k], down[k] = args[k] + h * dirn, args[k] - h * dirn
            slope = (loss(*up) - loss(*down)) / (2 * h)
            # the kernel's statistics are rounded to fp32: each moves xh by a few U relatively, hence the 2^-18 term
            scale = float((grad.abs() * dirn.abs()).sum())
            tol = float((bounds[k] * dirn.abs()).sum()) + 2.0 ** -18 * scale + 1e-6 * (1 + abs(slope))
            assert abs(float((grad * dirn).sum()) - slope) <= tol, (k, i)


def test_same_bits_twice_and_on_another_stream(cuda_lib):
    tg = cuda_lib
    x, dy = rows_of(23, 3000, 640, torch.bfloat16).cuda(), rows_of(24, 3000, 640, torch.bfloat16).cuda()
    w = rows_of(25, 1, 640, torch.bfloat16, shift=1.0)[0].cuda()
    y, mean, rstd = tg.layer_norm(x, w, stats=True)
    first = tg.layer_norm_backward(dy, x, mean, rstd, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = tg.layer_norm(x, w, stats=True, stream=side) + tg.layer_norm_backward(dy, x, mean, rstd, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip((y, mean, rstd) + first, again):
        assert torch.equal(a, b)


def test_graph_capture(cuda_lib):
    tg = cuda_lib
    x, dy = rows_of(26, 50, 256, torch.float32).cuda(), rows_of(27, 50, 256, torch.float32).cuda()
    want_y, mean, rstd = tg.layer_norm(x, stats=True)
    want = tg.layer_norm_backward(dy, x, mean, rstd)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, m, r = tg.layer_norm(x, stats=True)
        got = tg.layer_norm_backward(dy, x, m, r)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want_y) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rows,width", [(40, 72), (3, 8200), (3000, 1000), (2500, 333), (5, 20000), (700, 12000)])
@pytest.mark.parametrize("target", ["x", "dy"])
def test_results_in_place_of_inputs(cuda_lib, rows, width, target):
    """The C entry points with y in place of x, and dx in place of x or dy: the same bits, for every kernel."""
    tg = cuda_lib
    L = tg.load()
    x, dy = rows_of(35, rows, width, torch.float16).cuda(), rows_of(36, rows, width, torch.float16).cuda()
    w, b = rows_of(37, 1, width, torch.float16, shift=1.0)[0].cuda(), rows_of(38, 1, width, torch.float16)[0].cuda()
    y, mean, rstd = tg.layer_norm(x, w, b, stats=True)
    want = tg.layer_norm_backward(dy, x, mean, rstd, w)
    s = torch.cuda.current_stream().cuda_stream
    t = {"x": x.clone(), "dy": dy.clone()}
    dw, db = torch.empty_like(w), torch.empty_like(w)
    need = L.tgemm_layer_norm_workspace(rows, width)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert L.tgemm_layer_norm_backward(rows, width, tg.F16, tg.F16, t["dy"].data_ptr(), width, t["x"].data_ptr(), width,
                                       mean.data_ptr(), rstd.data_ptr(), w.data_ptr(), t[target].data_ptr(), width,
                                       dw.data_ptr(), db.data_ptr(), work.data_ptr(), need, s) == tg.OK
    for got, ref_ in zip((t[target], dw, db), want):
        assert torch.equal(got, ref_)
    z = x.clone()
    assert L.tgemm_layer_norm(rows, width, tg.F16, tg.F16, z.data_ptr(), width, w.data_ptr(), b.data_ptr(), 1e-5,
                              z.data_ptr(), width, None, None, s) == tg.OK
    assert torch.equal(z, y)


def test_refusals(cuda_lib):
    tg = cuda_lib
    x = torch.randn(4, 64, device="cuda")
    s = torch.ones(4, device="cuda")
    with pytest.raises(TypeError):
        tg.layer_norm(x.double())
    with pytest.raises(TypeError):
        tg.layer_norm(x, torch.ones(64, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        tg.layer_norm(x.cpu())
    with pytest.raises(ValueError):
        tg.layer_norm(x, torch.ones(63, device="cuda"))
    with pytest.raises(ValueError):
        tg.layer_norm(x.t())
    with pytest.raises(ValueError):
        tg.layer_norm(x[:1].expand(4, 64))
    with pytest.raises(ValueError):
        tg.layer_norm(x[:, :0])
    with pytest.raises(tg.TgemmError):
        tg.layer_norm(x, eps=-1.0)
    with pytest.raises(tg.TgemmError):
        tg.layer_norm(x, eps=float("nan"))
    with pytest.raises(ValueError):
        tg.layer_norm_backward(x[:2], x, s, s)
    with pytest.raises(TypeError):
        tg.layer_norm_backward(x.half(), x, s, s)
    with pytest.raises(TypeError):
        tg.layer_norm_backward(x, x, s.half(), s)
    with pytest.raises(ValueError):
        tg.layer_norm_backward(x, x, s[:3], s)


def test_c_abi_refusals(cuda_lib):
    tg = cuda_lib
    L = tg.load()
    x = torch.randn(4, 64, device="cuda")
    p = x.data_ptr()
    ok = (4, 64, tg.F32, tg.F32, p, 64, None, None, 1e-5, p, 64, None, None, None)

    def fwd(**change):
        names = ["rows", "width", "dtype", "wdtype", "x", "ldx", "w", "b", "eps", "y", "ldy", "mean", "rstd", "s"]
        a = dict(zip(names, ok))
        a.update(change)
        return L.tgemm_layer_norm(*[a[n] for n in names])

    assert fwd(rows=-1) == tg.ERR_INVALID_ARG
    assert fwd(width=0) == tg.ERR_INVALID_ARG
    assert fwd(ldx=63) == tg.ERR_INVALID_ARG
    assert fwd(ldy=63) == tg.ERR_INVALID_ARG
    assert fwd(x=None) == tg.ERR_INVALID_ARG
    assert fwd(y=None) == tg.ERR_INVALID_ARG
    assert fwd(dtype=7) == tg.ERR_UNSUPPORTED_DTYPE
    assert fwd(wdtype=tg.F16) == tg.ERR_UNSUPPORTED_DTYPE
    assert fwd(x=p + 2) == tg.ERR_ALIGNMENT
    assert fwd(rows=0, x=None, y=None) == tg.OK
    assert L.tgemm_layer_norm_workspace(4, 0) == -tg.ERR_INVALID_ARG
    bwd = (4, 64, tg.F32, tg.F32, p, 64, p, 64, p, p, None, p, 64, p, None)
    assert L.tgemm_layer_norm_backward(*bwd, None, 0, None) == tg.ERR_INVALID_ARG  # no workspace
    need = L.tgemm_layer_norm_workspace(4, 64)
    assert L.tgemm_layer_norm_backward(*bwd, p, need - 1, None) == tg.ERR_INVALID_ARG
