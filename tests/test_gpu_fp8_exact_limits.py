"""8-bit products with an operand just under 2 GiB whose sums are exact: codes of -1, 0
and 1 under scales that differ from row to row and from block to block, few enough of them
that every partial sum is a whole number below 2^24 (the eight products that an
8-bit instruction adds in fixed point have one size, so they lose nothing).  A wrong
row, block, scale or offset then shows in every output, whose only rounding is its type's."""
import pytest

import fp8_ref as f8
from test_gpu_fp8 import FD

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ONE = {"f8e4m3": 0x38, "f8e5m2": 0x3C}


@pytest.fixture(scope="module")
def ba():
    import conv_bias_activation_amd as m
    return m


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def operand(rows, K, fmt, block_rows, every, seed):
    """codes, scales: one value in `every` is 1 or -1, scales 1, 2, 4 or 8."""
    c, s = f8.shapes(rows, K, block_rows)
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.zeros(c, dtype=torch.uint8, device="cuda")
    for part in codes.split(max(1, 2 ** 27 // K)):
        r = torch.randint(0, 2 * every, part.shape, generator=g, device="cuda", dtype=torch.int16)
        part.copy_(torch.where(r == 0, ONE[fmt], torch.where(r == 1, ONE[fmt] | 0x80, 0)))
    if codes.shape[1] > K:
        codes[:, K:] = 0
    return codes.view(FD[fmt]), torch.randint(127, 131, s, generator=g, device="cuda", dtype=torch.uint8)


def values(codes, scales, rows, block_rows):
    """fp32 values of some rows."""
    b = codes.view(torch.uint8)[rows]
    v = torch.where(b == 0, 0.0, torch.where(b >= 128, -1.0, 1.0))
    at = torch.arange(codes.shape[0], device="cuda")[rows] // block_rows
    s = torch.exp2(scales[at].float() - 127).round()[:, :b.shape[1] // 128]
    return (v.view(len(b), -1, 128) * s[:, :, None]).view(len(b), -1)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("left", [True, False])
@pytest.mark.parametrize("rows,K,other,fmt,block_rows,every", [
    (32767, 65536, 40, "f8e4m3", 1, 16), (16383, 131072, 300, "f8e5m2", 128, 16), (1023, 2097152, 5, "f8e4m3", 1, 16), (2 ** 24 - 1, 100, 17, "f8e4m3", 128, 1),
    (131071, 16300, 130, "f8e5m2", 1, 4)])
def test_operand_of_two_gib(ba, rows, K, other, fmt, block_rows, every, left, out):
    big, small = operand(rows, K, fmt, block_rows, every, 0), operand(other, K, "f8e4m3", 1, 16, 1)
    M, N = (rows, other) if left else (other, rows)
    C = torch.full((M, N), 7.0, dtype=out, device="cuda")
    ba.gemm_fp8_bias_act(*(big if left else small), *(small if left else big), None, C)
    got = C if left else C.t()
    w = values(*small, slice(0, other), 1)
    # terms that are not zero: K / (every * 16) of them about, each 64 at most
    assert 1.5 * K / (every * 16) * 64 + 4096 < 2 ** 24
    step = max(1, 2 ** 28 // max(K, 128 * other))
    for i in range(0, rows, step):
        part = slice(i, min(i + step, rows))
        ref = torch.matmul(values(*big, part, block_rows), w.t().contiguous())
        assert torch.equal(got[part], ref.to(out)), (i, ba.last_tile_config())


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K,ahead", [(17000, 128, 4096, False), (20000, 100, 4000, False), (16300, 200, 4500, False), (10000, 300, 6800, True)])
def test_products_of_one_round_and_few_columns(ba, M, N, K, ahead, out):
    # operands of 64 MB and more; one or two columns of tiles have no wave ahead
    a, b = operand(M, K, "f8e4m3", 1, 4, 0), operand(N, K, "f8e5m2", 128, 4, 1)
    C = torch.full((M, N), 7.0, dtype=out, device="cuda")
    ba.gemm_fp8_bias_act(*a, *b, None, C)
    assert "4 stages" in ba.last_tile_config() and ("a wave ahead" in ba.last_tile_config()) == ahead
    one = torch.where(b[0].view(torch.uint8) == 0, 0.0, torch.where(b[0].view(torch.uint8) >= 128, -1.0, 1.0))
    s = torch.exp2(b[1].float() - 127).round()[torch.arange(N, device="cuda") // 128][:, :one.shape[1] // 128]
    w = (one.view(N, -1, 128) * s[:, :, None]).view(N, -1)
    assert torch.equal(C, torch.matmul(values(*a, slice(0, M), 1), w.t().contiguous()).to(out))
