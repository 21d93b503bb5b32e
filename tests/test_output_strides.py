"""The row operators' C entry points with outputs whose rows are apart from one
another, on and off the 16-byte boundary, between bands that must not change."""

import pytest
import torch

from tests import operator_reference as ref
from tests import test_norm
from tests.test_dropout import check

pytestmark = pytest.mark.gpu

DT = ref.DTYPES
GUARD = 512  # elements before and after
SENTINEL = 7.0


class Banded:
    """A [rows, width] matrix of row distance ld inside a buffer of sentinels; `shift` elements past a 16-byte boundary."""

    def __init__(self, rows, width, ld, dtype, values=None, shift=0):
        self.room = torch.full((GUARD + shift + rows * ld + GUARD,), SENTINEL, dtype=dtype, device="cuda")
        self.view = self.room[GUARD + shift:GUARD + shift + rows * ld].view(rows, ld)[:, :width]
        self.ld, self.ptr = ld, self.view.data_ptr()
        if values is not None:
            self.view.copy_(values)

    def untouched(self):
        rest = self.room.clone()
        start = self.view.storage_offset()
        rest[start:start + self.view.shape[0] * self.ld].view(-1, self.ld)[:, :self.view.shape[1]] = SENTINEL
        return bool((rest == SENTINEL).all())


def pads(dtype):
    """(row padding of the input, of the output, shift of the output) in elements; V fill 16 bytes."""
    v = 8 if dtype != "f32" else 4
    return [(0, 0, 0), (0, v, 0), (2 * v, v, 0), (3, 3 + v, 0), (1, 2, 0), (v, 0, 1), (0, 5, 3)]


SHAPES = [(1, 1), (5, 20000), (40, 72), (3, 8200), (300, 61), (2500, 333), (3000, 1000), (700, 8185), (320, 12288)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width", SHAPES)
def test_layer_norm(cuda_lib, rows, width, dtype):
    tg, dt = cuda_lib, DT[dtype]
    L, code = tg.load(), {"bf16": tg.BF16, "f32": tg.F32}[dtype]
    s = torch.cuda.current_stream().cuda_stream
    x, dy = test_norm.rows_of(51, rows, width, dt), test_norm.rows_of(52, rows, width, dt, shift=0.0)
    w, b = test_norm.rows_of(53, 1, width, dt, shift=1.0)[0], test_norm.rows_of(54, 1, width, dt)[0]
    wd, bd = w.cuda(), b.cuda()
    need = L.tgemm_layer_norm_workspace(rows, width)
    for pad_in, pad_out, shift in pads(dtype):
        gx, gdy = (Banded(rows, width, width + pad_in, dt, t) for t in (x, dy))
        gy, gdx = (Banded(rows, width, width + pad_out, dt, shift=shift) for _ in range(2))
        mean, rstd = (Banded(1, rows, rows, torch.float32) for _ in range(2))
        dw, db = (Banded(1, width, width, dt) for _ in range(2))
        work = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")
        what = f"paddings {pad_in} and {pad_out}, shift {shift}: "
        assert L.tgemm_layer_norm(rows, width, code, code, gx.ptr, gx.ld, wd.data_ptr(), bd.data_ptr(), 1e-5, gy.ptr, gy.ld,
                                  mean.ptr, rstd.ptr, s) == tg.OK
        test_norm.check_forward(x, w, b, (gy.view, mean.view[0], rstd.view[0]))
        assert L.tgemm_layer_norm_backward(rows, width, code, code, gdy.ptr, gdy.ld, gx.ptr, gx.ld, mean.ptr, rstd.ptr,
                                           wd.data_ptr(), gdx.ptr, gdx.ld, dw.ptr, db.ptr, work.data_ptr(), need, s) == tg.OK
        args = (dy, x, mean.view[0].cpu(), rstd.view[0].cpu(), w)
        for name, g, r, bound in zip(("dx", "dweight", "dbias"), (gdx.view, dw.view[0], db.view[0]),
                                     ref.layer_norm_backward(*args), ref.layer_norm_backward_bounds(*args)):
            test_norm.within(g, r, bound, what + name)
        assert all(t.untouched() for t in (gx, gdy, gy, gdx, mean, rstd, dw, db)), what
        assert bool((work[need:] == 77).all()), what


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [1, 3, 7, 8, 9, 255, 2047, 2049, 5003])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_dropout(cuda_lib, n, shift, dtype):
    tg, dt = cuda_lib, DT[dtype]
    L, code = tg.load(), {"bf16": tg.BF16, "f16": tg.F16, "f32": tg.F32}[dtype]
    s = torch.cuda.current_stream().cuda_stream
    gen = torch.Generator().manual_seed(n)
    x, res = torch.randn(n, generator=gen).to(dt), torch.randn(n, generator=gen).to(dt)
    gx, gr = (Banded(1, n, n, dt, t, shift) for t in (x, res))
    for r in (None, gr):
        gy = Banded(1, n, n, dt, shift=shift)
        assert L.tgemm_dropout(n, code, gx.ptr, r.ptr if r else None, gy.ptr, 0.4, 5, 6, s) == tg.OK
        check(gy.view[0], x, res if r else None, 0.4, 5, 6)
        assert gy.untouched() and gx.untouched() and gr.untouched()
    for p in (1.0, 0.0):
        gy = Banded(1, n, n, dt, shift=shift)
        assert L.tgemm_dropout(n, code, gx.ptr, gr.ptr, gy.ptr, p, 5, 6, s) == tg.OK
        check(gy.view[0], x, res, p, 5, 6)
        assert gy.untouched()
