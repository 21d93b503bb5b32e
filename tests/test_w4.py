"""Products with 4-bit weights against the 64-bit definition.

Bound: q - z is exact; a group's fp32 sum and the sums over groups and warps are
off by at most 2 U a tensor-core step of 16 (and 16 terms aligned within one),
U a group for its scaled sum, 8 U for the warps', of the sum of magnitudes; then
the output's rounding."""

import pytest
import torch

from tests import expert_reference as exp
from tests import operator_reference as ref

DT = ref.DTYPES
U = ref.U


def make(seed, rows, width, group, dtype, zeros=False, experts=None, scale_dtype=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lead = () if experts is None else (experts,)
    packed = torch.randint(0, 256, (*lead, rows, width // 2), dtype=torch.uint8, device="cuda", generator=gen)
    scales = (0.01 + 0.02 * torch.rand(*lead, rows, width // group, device="cuda", generator=gen)).to(scale_dtype or DT[dtype])
    z = torch.randint(0, 16, scales.shape, dtype=torch.uint8, device="cuda", generator=gen) if zeros else None
    return packed, scales, z


def rows_of(seed, *shape, dtype):
    gen = torch.Generator(device="cuda").manual_seed(seed + 1000)
    return torch.randn(*shape, device="cuda", generator=gen).to(DT[dtype])


def within(got, x, w, group, what=""):
    """got [..., rows] against x [..., width] and w [rows, width]."""
    want, mag = x.double() @ w.T, x.double().abs() @ w.abs().T
    k = x.shape[-1]
    bound = (2 * (group / 16 + 16) + 2 * k / group + 16) * U * mag + 1.01 * ref.u_out(got.dtype) * want.abs() + ref.tiny(got.dtype)
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), f"{what}: worst error/bound {float((off / bound).max()):.3g}"


SIZES = [(1, 32, 32), (5, 64, 32), (16, 96, 96), (17, 128, 128), (33, 2048, 32), (100, 640, 64), (77, 1024, 128), (250, 4096, 256),
         (40, 1280, 1280), (1000, 320, 160), (31, 8192, 128), (515, 192, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("size", SIZES)
def test_sizes(cuda_lib, size, zeros, dtype):
    rows, width, group = size
    packed, scales, z = make(sum(size), rows, width, group, dtype, zeros)
    w = exp.unpack_w4(packed, scales, z)
    for tokens in (1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 70):
        x = rows_of(tokens, tokens, width, dtype=dtype)
        y = cuda_lib.gemm_w4(x, packed, scales, z)
        assert y.shape == (tokens, rows) and y.dtype == x.dtype
        within(y, x, w, group, f"{tokens} tokens")
        y32 = cuda_lib.gemm_w4(x, packed, scales, z, out_dtype=torch.float32)
        within(y32, x, w, group, f"{tokens} tokens, fp32")
        assert torch.equal(y32.to(x.dtype), y)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("width,group", [(256, 128), (320, 64), (416, 32), (8192, 32)])
def test_many_rows_of_weights(cuda_lib, width, group, dtype):
    """More rows than one block of 32 on each multiprocessor takes, and a number that no block's size divides."""
    packed, scales, z = make(width, 5003, width, group, dtype, True)
    w = exp.unpack_w4(packed, scales, z)
    for tokens in (1, 10, 17, 32, 45):
        x = rows_of(tokens, tokens, width, dtype=dtype)
        within(cuda_lib.gemm_w4(x, packed, scales, z, out_dtype=torch.float32), x, w, group, f"{tokens} tokens")


@pytest.mark.gpu
def test_many_rows_of_experts(cuda_lib):
    packed, scales, z = make(6, 1100, 256, 64, "bf16", True, 5)
    e = torch.randint(-1, 6, (60, 2), generator=torch.Generator().manual_seed(6)).int().cuda()
    x = rows_of(6, 60, 256, dtype="bf16")
    y = cuda_lib.gemm_w4(x, packed, scales, z, experts=e)
    for i in range(5):
        t, j = (e == i).nonzero(as_tuple=True)
        within(y[t, j], x[t], exp.unpack_w4(packed[i], scales[i], z[i]), 64, f"expert {i}")
    assert not y[(e < 0) | (e > 4)].any()


@pytest.mark.gpu
def test_a_row_does_not_depend_on_its_batch(cuda_lib):
    packed, scales, z = make(1, 300, 1024, 64, "bf16", True)
    x = rows_of(1, 40, 1024, dtype="bf16")
    y = cuda_lib.gemm_w4(x, packed, scales, z)
    for i in (0, 7, 8, 31, 39):
        assert torch.equal(cuda_lib.gemm_w4(x[i:i + 1], packed, scales, z), y[i:i + 1])


@pytest.mark.gpu
def test_scales_of_fp32_and_shapes_of_x(cuda_lib):
    packed, scales, z = make(2, 90, 512, 128, "bf16", True, scale_dtype=torch.float32)
    w = exp.unpack_w4(packed, scales, z)
    x = rows_of(2, 3, 4, 512, dtype="bf16")
    y = cuda_lib.gemm_w4(x, packed, scales, z)
    assert y.shape == (3, 4, 90)
    within(y, x, w, 128)
    assert torch.equal(cuda_lib.gemm_w4(x[1, 2], packed, scales, z), y[1, 2])  # a vector
    wide = torch.full((12, 640), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 64:576] = x.reshape(12, 512)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    apart = cuda_lib.gemm_w4(wide[:, 64:576], packed, scales, z, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(apart, y.reshape(12, 90))
    assert cuda_lib.gemm_w4(x[:0], packed, scales, z).shape == (0, 4, 90)


@pytest.mark.gpu
def test_every_nibble_and_zero_point(cuda_lib):
    """One-hot rows read single weights: (q - z) s is exact in fp32 but for its rounding."""
    packed = torch.arange(256, dtype=torch.uint8, device="cuda").reshape(16, 16)
    packed = torch.cat([packed] * 2, 1).repeat(16, 1).contiguous()  # 256 rows of 64 weights
    zeros = torch.arange(16, dtype=torch.uint8, device="cuda").repeat_interleave(16)[:, None].repeat(1, 2).contiguous()
    scales = (torch.rand(256, 2, device="cuda") + 0.5).half()
    w = exp.unpack_w4(packed, scales, zeros)
    y = cuda_lib.gemm_w4(torch.eye(64, device="cuda").half(), packed, scales, zeros, out_dtype="f32")
    assert torch.equal(y.double(), w.T)
    wb = exp.unpack_w4(packed, scales.bfloat16(), zeros)
    y = cuda_lib.gemm_w4(torch.eye(64, device="cuda").bfloat16(), packed, scales.bfloat16(), zeros, out_dtype=torch.float32)
    assert torch.equal(y.double(), wb.T)


@pytest.mark.gpu
def test_infinities_and_nans_stay_in_their_rows(cuda_lib):
    packed, scales, _ = make(3, 64, 256, 64, "f16")
    x = rows_of(3, 12, 256, dtype="f16")
    x[3, 17], x[5, 200] = float("nan"), float("inf")
    y = cuda_lib.gemm_w4(x, packed, scales)
    ok = torch.ones(12, dtype=torch.bool, device="cuda")
    ok[3] = ok[5] = False
    assert bool(y[3].isnan().all()) and not y[5].isfinite().any()
    within(y[ok], x[ok], exp.unpack_w4(packed, scales, None), 64)


# ------------------------------------------------------------------ a matrix for each pair

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,top,experts", [(1, 1, 1), (1, 4, 8), (4, 4, 32), (6, 2, 3), (9, 1, 2), (40, 2, 5), (70, 3, 3), (3, 8, 24)])
def test_experts(cuda_lib, tokens, top, experts, dtype):
    rows, width, group = 84, 384, 64
    packed, scales, z = make(tokens, rows, width, group, dtype, True, experts)
    w = exp.unpack_w4(packed, scales, z)
    gen = torch.Generator().manual_seed(tokens)
    chosen = torch.stack([torch.randperm(max(experts, top), generator=gen)[:top] for _ in range(tokens)]).int().cuda()
    if tokens > 5:  # not routed, and the same one twice
        chosen[2, 0], chosen[3, top - 1], chosen[4] = -1, experts, int(chosen[4, 0])
    for x in (rows_of(7, tokens, width, dtype=dtype), rows_of(8, tokens, top, width, dtype=dtype)):
        y = cuda_lib.gemm_w4(x, packed, scales, z, experts=chosen)
        assert y.shape == (tokens, top, rows)
        for t in range(tokens):
            for j in range(top):
                e = int(chosen[t, j])
                if not 0 <= e < experts:
                    assert not y[t, j].any()
                    continue
                within(y[t, j], x[t] if x.dim() == 2 else x[t, j], w[e], group, f"{t}, {j}")


@pytest.mark.gpu
def test_matrices_beyond_32_bits_of_bytes(cuda_lib):
    """The last expert's matrix starts behind 2^32 bytes."""
    experts, rows, width = 34, 8192, 32768  # 128 MiB a matrix
    packed = torch.zeros(experts, rows, width // 2, dtype=torch.uint8, device="cuda")
    packed[33] = torch.randint(0, 256, (rows, width // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((experts, rows, 1), 0.02, dtype=torch.bfloat16, device="cuda")
    x = rows_of(4, 1, width, dtype="bf16")
    y = cuda_lib.gemm_w4(x, packed, scales, experts=torch.tensor([[33, 0]], dtype=torch.int32, device="cuda"))
    pick = slice(8000, 8192)
    within(y[0, 0, pick], x[0], exp.unpack_w4(packed[33, pick], scales[33, pick], None), width)
    within(y[0, 1, pick], x[0], exp.unpack_w4(packed[0, pick], scales[0, pick], None), width)


@pytest.mark.gpu
def test_captured(cuda_lib):
    packed, scales, _ = make(9, 200, 512, 128, "bf16", experts=6)
    x, chosen = rows_of(9, 5, 512, dtype="bf16"), torch.randint(0, 6, (5, 2), dtype=torch.int32, device="cuda")
    cuda_lib.gemm_w4(x, packed, scales, experts=chosen)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = cuda_lib.gemm_w4(x, packed, scales, experts=chosen)
    for seed in (1, 2):
        x.copy_(rows_of(seed, 5, 512, dtype="bf16"))
        chosen.copy_(torch.randint(0, 6, (5, 2), dtype=torch.int32))
        graph.replay()
        assert torch.equal(y, cuda_lib.gemm_w4(x, packed, scales, experts=chosen))


def test_refusals_without_a_gpu():
    import software_pipelined_tiled_02_gb300 as tg

    with pytest.raises(ValueError, match="CUDA tensor"):
        tg.gemm_w4(torch.zeros(2, 32).half(), torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1).half())
    L = tg.load()
    call = lambda **k: L.tgemm_gemm_fourbit(*{"p": 4, "n": 8, "k": 64, "g": 32, "dt": tg.BF16, "x": None, "ld": 64, "each": 1, "w": None,  # noqa: E731
                                         "s": None, "sdt": tg.F32, "z": None, "e": None, "ne": 1, "y": None, "ydt": tg.BF16,
                                         "st": None, **k}.values())
    for bad in ({"dt": tg.F32}, {"sdt": tg.F16}, {"ydt": tg.F16}, {"dt": 9}):
        assert call(**bad) == tg.ERR_UNSUPPORTED_DTYPE, bad
    for bad in ({"p": -1}, {"p": (1 << 20) + 1}, {"n": 0}, {"k": 0}, {"g": 16}, {"g": 48}, {"g": 0}, {"k": 96, "g": 64}, {"each": 0},
                {"each": 3}, {"ne": 0}, {"ne": 2}, {"ne": 65535, "e": 4}):
        assert call(**bad) == tg.ERR_INVALID_ARG, bad


@pytest.mark.gpu
def test_refusals(cuda_lib):
    tg = cuda_lib
    packed, scales, z = make(1, 8, 64, 32, "bf16", True)
    x = rows_of(1, 4, 64, dtype="bf16")
    e = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for bad in ((x.float(), packed, scales), (x.half(), packed, scales), (x, packed.int(), scales), (x, packed, scales, z.int()),
                (x, packed[None], scales[None], None, e.long())):
        with pytest.raises(TypeError):
            tg.gemm_w4(*bad)
    with pytest.raises(TypeError):
        tg.gemm_w4(x, packed, scales, out_dtype=torch.float16)
    for bad in ((x[:, :32], packed, scales), (x, packed.t(), scales), (x, packed[:4], scales), (x, packed, scales[:, :1].expand(8, 4)),
                (x, packed, scales, z[:4]), (x.cpu(), packed, scales), (x, packed.cpu(), scales), (x, packed, scales, None, e),
                (x, packed[None], scales[None], None, e[:3]), (x, packed[None], scales[None], None, e[0]),
                (x, packed[None], scales[None]), (x, packed, torch.zeros(8, 4, device="cuda").bfloat16())):
        with pytest.raises(ValueError):
            tg.gemm_w4(*bad)
    off = torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 64)
    with pytest.raises(tg.TgemmError) as err:
        tg.gemm_w4(off, packed, scales)
    assert err.value.code == tg.ERR_ALIGNMENT


def test_types_that_the_library_does_not_have():
    import software_pipelined_tiled_02_gb300 as tg

    w = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1).half()
    for x in (torch.zeros(2, 32).half(), torch.zeros(2, 32).long(), torch.zeros(2, 32).double(), [1.0]):
        for out in (torch.float64, "f64", torch.bfloat16):
            with pytest.raises((TypeError, ValueError)):
                tg.gemm_w4(x, *w, out_dtype=out)
    with pytest.raises(TypeError, match="out_dtype"):
        tg.gemm_w4(torch.zeros(2, 32).half(), *w, out_dtype=torch.float64)
