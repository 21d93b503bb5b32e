"""Outputs of the mixture-of-experts operators through the C entry points, with bands around them and between their
rows; strides, scales and numbers of matrices that the other tests leave out."""

import pytest
import torch

from tests import expert_reference as exp
from tests import test_experts, test_route, test_w4

pytestmark = pytest.mark.gpu
BAND = 64


def banded(rows, ld, dtype):
    """A buffer of 7s and the rows inside it."""
    t = torch.full(((rows + 2 * BAND) * ld,), 7, dtype=dtype, device="cuda")
    return t, t[BAND * ld:-BAND * ld].view(rows, ld)


def only(t, inner, want):
    """`want` stands in the first columns of `inner`, and everything else is as it was."""
    assert torch.equal(inner[:, :want.shape[1]], want)
    inner[:, :want.shape[1]] = 7
    assert bool((t == 7).all())


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,experts,top,width,hidden", [(1, 6, 4, 72, 136), (1, 1, 1, 8, 8), (1, 40, 32, 264, 72), (2, 9, 2, 72, 264),
                                                             (12, 40, 8, 520, 136), (90, 7, 3, 72, 136), (600, 7, 3, 136, 72)])
def test_served_tokens(cuda_lib, tokens, experts, top, width, hidden, dtype):
    tg, d = cuda_lib, test_experts.make(tokens, tokens, experts, min(top, experts), width, hidden, dtype, invalid=tokens > 1)
    L, plan, top = tg.load(), tg.GatedFFN(width, hidden, dtype), min(top, experts)
    need = L.tgemm_experts_workspace(plan.handle, tokens, experts, top, 0)
    work = torch.zeros(need + 512, dtype=torch.uint8, device="cuda")
    weights = [v for k in ("wg", "wu", "wd") for v in (d[k].data_ptr(), d[k].stride(1), d[k].stride(0))]
    want = tg.expert_ffn(*test_experts.args(d))
    for ld in (width, width + 8):
        t, y = banded(tokens, ld, d["x"].dtype)
        assert L.tgemm_experts_forward(plan.handle, tokens, experts, top, d["x"].data_ptr(), width, d["e"].data_ptr(), d["w"].data_ptr(),
                                       *weights, y.data_ptr(), ld, None, None, None, work.data_ptr(), need, stream()) == tg.OK
        torch.cuda.synchronize()
        only(t, y, want)
        assert not work[need:].any()
    assert plan.status()[0] == tg.OK
    plan.close()


def test_dx_with_distant_rows(cuda_lib):
    tokens, experts, top, width, hidden = 150, 6, 2, 72, 136
    tg, d = cuda_lib, test_experts.make(1, tokens, experts, top, width, hidden, "bf16", invalid=True)
    L, plan = tg.load(), tg.GatedFFN(width, hidden)
    need = L.tgemm_experts_workspace(plan.handle, tokens, experts, top, 2)
    work = torch.zeros(need + 512, dtype=torch.uint8, device="cuda")
    weights = [v for k in ("wg", "wu", "wd") for v in (d[k].data_ptr(), d[k].stride(1), d[k].stride(0))]
    _, saved = tg.expert_ffn(*test_experts.args(d), save=True)
    want = tg.expert_ffn_backward(d["dy"], *test_experts.args(d), saved)[0]
    t, dx = banded(tokens, width + 8, torch.bfloat16)
    assert L.tgemm_experts_backward(plan.handle, tokens, experts, top, d["dy"].data_ptr(), width, d["x"].data_ptr(), width,
                                    d["e"].data_ptr(), d["w"].data_ptr(), *weights, *(s.data_ptr() for s in saved), dx.data_ptr(), width + 8,
                                    None, None, None, None, work.data_ptr(), need, stream()) == tg.OK
    torch.cuda.synchronize()
    only(t, dx, want)
    assert not work[need:].any() and plan.status()[0] == tg.OK
    plan.close()


@pytest.mark.parametrize("tokens", [1, 3, 40, 400])
def test_experts_a_few_elements_apart(cuda_lib, tokens):
    """All weights of an expert in one block, of a size that no row's length divides."""
    d = test_experts.make(2, tokens, 9, 2, 136, 264, "bf16")
    want_y, saved = cuda_lib.expert_ffn(*test_experts.args(d), save=True)
    served = cuda_lib.expert_ffn(*test_experts.args(d))
    want = cuda_lib.expert_ffn_backward(d["dy"], *test_experts.args(d), saved)
    size = 136 * 264
    blocks = torch.full((9, 3 * size + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    for i, k in enumerate(("wg", "wu", "wd")):
        part = blocks[:, i * size:(i + 1) * size].view(9, *d[k].shape[1:])
        part.copy_(d[k])
        d[k] = part
    assert d["wg"].stride(0) == 3 * size + 8
    y, saved = cuda_lib.expert_ffn(*test_experts.args(d), save=True)
    assert torch.equal(y, want_y) and torch.equal(cuda_lib.expert_ffn(*test_experts.args(d)), served)
    assert all(torch.equal(a, b) for a, b in zip(cuda_lib.expert_ffn_backward(d["dy"], *test_experts.args(d), saved), want))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tokens,experts,top", [(1, 1, 1), (3, 7, 2), (5, 33, 6), (9, 128, 8), (7, 257, 32), (2, 1024, 5)])
def test_choices_and_gradients(cuda_lib, tokens, experts, top, dtype):
    tg, L = cuda_lib, cuda_lib.load()
    logits, bias = (t.cuda() for t in test_route.make(3, tokens, experts, dtype))
    code = {"f16": tg.F16, "bf16": tg.BF16, "f32": tg.F32}[dtype]
    for b in (None, bias):
        want = tg.route(logits, top, "sigmoid", bias=b)
        (tw, w), (te, e) = banded(tokens, top, torch.float32), banded(tokens, top, torch.int32)
        assert L.tgemm_route(tokens, experts, top, code, logits.data_ptr(), experts, b.data_ptr() if b is not None else None, 1, 1, 1, 1, 1,
                             1.0, w.data_ptr(), e.data_ptr(), stream()) == tg.OK
        torch.cuda.synchronize()
        only(tw, w, want[0])
        only(te, e, want[1])
    for scoring, name in ((0, "softmax"), (1, "sigmoid")):
        for renormalize in (0, 1):
            t, dl = banded(tokens, experts, logits.dtype)
            assert L.tgemm_route_backward(tokens, experts, top, code, want[0].data_ptr(), logits.data_ptr(), experts, want[1].data_ptr(),
                                          scoring, renormalize, 1.0, dl.data_ptr(), stream()) == tg.OK
            torch.cuda.synchronize()
            only(t, dl, tg.route_backward(want[0], logits, want[1], name, renormalize=bool(renormalize)))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,width,group", [(1, 32, 32), (77, 320, 64), (1003, 256, 128), (9999, 64, 32)])
@pytest.mark.parametrize("experts", [None, 3])
def test_products(cuda_lib, experts, rows, width, group, dtype):
    tg, L = cuda_lib, cuda_lib.load()
    packed, scales, z = test_w4.make(rows, rows, width, group, dtype, True, experts)
    code = tg.BF16 if dtype == "bf16" else tg.F16
    for pairs in (1, 9, 30, 50):
        x = test_w4.rows_of(pairs, pairs, width, dtype=dtype)
        e = None
        if experts:
            e = torch.randint(-1, experts + 1, (pairs, 1), generator=torch.Generator().manual_seed(pairs)).int().cuda()
        for out, out_code in ((x.dtype, code), (torch.float32, tg.F32)):
            want = tg.gemm_w4(x, packed, scales, z, experts=e, out_dtype=out).view(pairs, rows)
            t, y = banded(pairs, rows, out)
            assert L.tgemm_gemm_fourbit(pairs, rows, width, group, code, x.data_ptr(), width, 1, packed.data_ptr(), scales.data_ptr(), code,
                                        z.data_ptr(), e.data_ptr() if experts else None, experts or 1, y.data_ptr(), out_code,
                                        stream()) == tg.OK
            torch.cuda.synchronize()
            only(t, y, want)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("rows,width,group", [(70, 16384, 32), (5003, 16384, 32), (40, 40960, 64), (33, 65536, 128)])
def test_products_with_more_scales_than_shared_memory_holds(cuda_lib, rows, width, group, zeros, dtype):
    packed, scales, z = test_w4.make(5, rows, width, group, dtype, zeros)
    w = exp.unpack_w4(packed, scales, z)
    for tokens in (1, 3, 8, 12, 25, 40):
        x = test_w4.rows_of(tokens, tokens, width, dtype=dtype)
        test_w4.within(cuda_lib.gemm_w4(x, packed, scales, z), x, w, group, f"{tokens} tokens")
    if rows < 100:
        stacked = [torch.stack([t, t.flip(0)]) if t is not None else None for t in (packed, scales, z)]
        x = test_w4.rows_of(6, 6, width, dtype=dtype)
        e = torch.tensor([[0, 1], [1, 2], [0, 0], [-1, 1], [1, 0], [0, 1]], dtype=torch.int32, device="cuda")
        y = cuda_lib.gemm_w4(x, *stacked, experts=e)
        for i, matrix in enumerate((w, w.flip(0))):
            t, j = (e == i).nonzero(as_tuple=True)
            test_w4.within(y[t, j], x[t], matrix, group, f"expert {i}")
        assert not y[(e < 0) | (e > 1)].any()


def test_products_with_as_many_matrices_as_there_may_be(cuda_lib):
    packed, scales, _ = test_w4.make(7, 3, 32, 32, "bf16", False, 65534)
    x = test_w4.rows_of(7, 200, 32, dtype="bf16")
    gen = torch.Generator().manual_seed(7)
    e = torch.randint(0, 65534, (200, 2), generator=gen).int().cuda()
    e[:2, 0], e[2, 0], e[3, 0] = 65533, 65534, -1
    y = cuda_lib.gemm_w4(x, packed, scales, experts=e)
    ok = (e >= 0) & (e < 65534)
    w = exp.unpack_w4(packed, scales, None)[e.clamp(0, 65533).long()]
    want = (w @ x.double()[:, None, :, None])[..., 0]
    mag = (w.abs() @ x.double().abs()[:, None, :, None])[..., 0]
    bound = 64 * test_w4.U * mag + 1.01 * 2.0 ** -8 * want.abs()  # two steps and one group (8 U), and the rounding to bf16
    assert bool(((y.double() - want).abs() <= bound)[ok].all()) and not y[~ok].any()
    # more pairs than matrices: a slot for each matrix and one for those that name none
    e = torch.cat([torch.arange(65534), torch.tensor([-1, 65534, 5])]).int().cuda()[:, None]
    x = test_w4.rows_of(8, len(e), 32, dtype="bf16")
    y = cuda_lib.gemm_w4(x, packed, scales, experts=e)[:, 0]
    w = exp.unpack_w4(packed, scales, None)[e.clamp(0, 65533).long()[:, 0]]
    want, mag = (w @ x.double()[:, :, None])[..., 0], (w.abs() @ x.double().abs()[:, :, None])[..., 0]
    ok = (e[:, 0] >= 0) & (e[:, 0] < 65534)
    assert bool(((y.double() - want).abs() <= 64 * test_w4.U * mag + 1.01 * 2.0 ** -8 * want.abs())[ok].all()) and not y[~ok].any()
