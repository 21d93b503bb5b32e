"""Dropout with a computed mask: the generator against its published test
vectors (CPU), and the GPU kernel against the 64-bit definition."""

import numpy as np
import pytest
import torch

from tests import operator_reference as ref

DT = ref.DTYPES


def test_reference_generator_against_published_vectors():
    """Known answers of Philox4x32-10 from the authors' distribution."""
    f = 0xFFFFFFFF
    assert ref.philox4x32((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ref.philox4x32((f, f, f, f), (f, f)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert ref.philox4x32((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def expected(x, res, p, seed, offset):
    kept = torch.from_numpy(ref.dropout_kept(0, x.numel(), p, seed, offset)).reshape(x.shape)
    y = torch.where(kept, x.double() / (1 - p) if p < 1 else x.double() * 0, torch.zeros((), dtype=torch.float64))
    return kept, y if res is None else y + res.double()


def check(got, x, res, p, seed, offset):
    kept, want = expected(x, res, p, seed, offset)
    got = got.cpu()
    if res is None:
        assert torch.equal(got != 0, kept & (x != 0))
    # 1/(1-p), the product and the sum are rounded to fp32, then once to the output type
    mag = x.double().abs() / (1 - p if p < 1 else 1) + (res.double().abs() if res is not None else 0)
    bound = 4 * ref.U * mag + ref.u_out(x.dtype) * want.abs() * 1.01 + ref.tiny(x.dtype)
    assert bool(((got.double() - want).abs() <= bound).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [0, 1, 3, 4, 5, 8, 9, 1001, 4099])
@pytest.mark.parametrize("residual", [False, True])
def test_against_definition(cuda_lib, n, dtype, residual):
    gen = torch.Generator().manual_seed(n)
    x = torch.randn(n, generator=gen).to(DT[dtype])
    res = torch.randn(n, generator=gen).to(DT[dtype]) if residual else None
    seed, offset = 0xFEDCBA9876543210 + n, (1 << 40) + 77
    y = cuda_lib.dropout(x.cuda(), 0.3, seed, offset, residual=res.cuda() if residual else None)
    check(y, x, res, 0.3, seed & (1 << 64) - 1, offset)


@pytest.mark.gpu
@pytest.mark.parametrize("p", [0.0, 2.0 ** -32, 0.5, 1.0 - 2.0 ** -32, 1.0])
def test_probabilities(cuda_lib, p):
    x = torch.randn(3000, generator=torch.Generator().manual_seed(1))
    y = cuda_lib.dropout(x.cuda(), p, 11, 12)
    check(y, x, None, p, 11, 12)
    if p == 0:
        assert torch.equal(y.cpu(), x)
    if p == 1:
        assert not y.any()
        res = torch.randn(3000, generator=torch.Generator().manual_seed(2)).cuda()
        assert torch.equal(cuda_lib.dropout(x.cuda(), p, 11, 12, residual=res), res)


@pytest.mark.gpu
def test_backward_meets_the_forward_mask_and_shapes_do_not_matter(cuda_lib):
    tg = cuda_lib
    x = torch.ones(37, 129, device="cuda")
    y = tg.dropout(x, 0.25, 5, 6)
    assert torch.equal(y, tg.dropout_backward(x, 0.25, 5, 6))
    assert torch.equal(y.flatten(), tg.dropout(x.flatten(), 0.25, 5, 6))
    assert torch.equal(y.half() != 0, tg.dropout(x.half(), 0.25, 5, 6) != 0)
    assert not torch.equal(y, tg.dropout(x, 0.25, 5, 7)) and not torch.equal(y, tg.dropout(x, 0.25, 6, 6))
    off = torch.ones(37 * 129 + 1, device="cuda")[1:]  # off the 16-byte boundary
    assert torch.equal(tg.dropout(off, 0.25, 5, 6), y.flatten())


@pytest.mark.gpu
def test_share_of_kept_elements(cuda_lib):
    n, p = 1 << 22, 0.1
    kept = float((cuda_lib.dropout(torch.ones(n, device="cuda"), p, 123, 0) != 0).double().mean())
    assert abs(kept - (1 - p)) < 6 * (p * (1 - p) / n) ** 0.5  # six standard deviations


@pytest.mark.gpu
def test_dropped_infinities_and_nans(cuda_lib):
    x = torch.full((4096,), float("nan"))
    x[::2] = float("inf")
    y = cuda_lib.dropout(x.cuda(), 0.5, 3, 4).cpu()
    kept = torch.from_numpy(ref.dropout_kept(0, 4096, 0.5, 3, 4))
    assert not y[~kept].any()
    assert bool(y[kept & x.isnan()].isnan().all()) and bool((y[kept & ~x.isnan()] == float("inf")).all())


@pytest.mark.gpu
def test_more_elements_than_32_bits_count(cuda_lib):
    """The block index passes into the counter's second word at element 2^34; the element index passes 2^32 here."""
    n = (1 << 32) + 13
    x = torch.ones(n, dtype=torch.float16, device="cuda")
    y = cuda_lib.dropout(x, 0.5, 21, 22)
    for first in (0, (1 << 31) - 5, (1 << 32) - 7, n - 40):
        kept = ref.dropout_kept(first, 40 if first + 40 <= n else n - first, 0.5, 21, 22)
        assert np.array_equal((y[first:first + len(kept)] != 0).cpu().numpy(), kept)


@pytest.mark.gpu
def test_another_stream(cuda_lib):
    x = torch.randn(100003, device="cuda").half()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = cuda_lib.dropout(x, 0.1, 1, 2, residual=x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, cuda_lib.dropout(x, 0.1, 1, 2, residual=x))


@pytest.mark.gpu
def test_refusals(cuda_lib):
    tg = cuda_lib
    x = torch.randn(8, 8, device="cuda")
    with pytest.raises(TypeError):
        tg.dropout(x.double(), 0.1, 0)
    with pytest.raises(ValueError):
        tg.dropout(x.cpu(), 0.1, 0)
    with pytest.raises(ValueError):
        tg.dropout(x.t(), 0.1, 0)
    for p in (-0.1, 1.1, float("nan")):
        with pytest.raises(ValueError):
            tg.dropout(x, p, 0)
    with pytest.raises(ValueError):
        tg.dropout(x, 0.1, 0, residual=x[:4])
    with pytest.raises(TypeError):
        tg.dropout(x, 0.1, 0, residual=x.half())
    L, p = tg.load(), x.data_ptr()
    assert L.tgemm_dropout(-1, tg.F32, p, None, p, 0.1, 0, 0, None) == tg.ERR_INVALID_ARG
    assert L.tgemm_dropout(4, tg.F32, p, None, p, 1.5, 0, 0, None) == tg.ERR_INVALID_ARG
    assert L.tgemm_dropout(4, tg.F32, None, None, p, 0.1, 0, 0, None) == tg.ERR_INVALID_ARG
    assert L.tgemm_dropout(4, 9, p, None, p, 0.1, 0, 0, None) == tg.ERR_UNSUPPORTED_DTYPE
    assert L.tgemm_dropout(4, tg.F32, p + 2, None, p, 0.1, 0, 0, None) == tg.ERR_ALIGNMENT
    assert L.tgemm_dropout(0, tg.F32, None, None, None, 0.1, 0, 0, None) == tg.OK
