"""Column sums of bias_act_grad and layer_norm_grad over small whole numbers:
fp32 holds every partial sum, so that the result is the whole number itself in any
order of additions, and a row that is left out or added twice shows.  From one row to
tensors just under 2 GiB, and rows past the length that is read again."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ba():
    import conv_bias_activation_amd as m
    return m


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def whole(M, N, dt, lo, hi, seed):
    """[M, N] of whole numbers lo .. hi."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty((M, N), dtype=dt, device="cuda")
    for part in out.split(max(1, 2 ** 27 // N)):
        part.copy_(torch.randint(lo, hi + 1, part.shape, generator=g, device="cuda", dtype=torch.int8))
    return out


def check(got, f, M, N):
    """got [N] against the sums of f(rows) in 64 bits."""
    ref = torch.zeros(N, dtype=torch.float64, device="cuda")
    for i in range(0, M, max(1, 2 ** 25 // N)):
        ref += f(slice(i, i + max(1, 2 ** 25 // N))).sum(0)
    assert float(ref.abs().max()) < 2 ** 24              # (the terms are of both signs, so partial sums stay far below too)
    bad = got.double() != ref
    assert not bool(bad.any()), (int(bad.sum()), got[bad][:3].tolist(), ref[bad][:3].tolist())


# M * (the largest term) stays below 2^24, so every partial sum does
ACT = [(1, 1, F32), (1, 4096, BF16), (3, 7, F16), (300, 1003, BF16), (5000, 24, F32), (70000, 3, BF16), (4097, 520, F16), (8192, 16384, BF16),
       (32767, 16384, F32), (2 ** 23 - 1, 128, BF16), (2 ** 23 - 1, 9, F32), (3, 357913939, BF16)]


@pytest.mark.parametrize("M,N,dt", ACT)
def test_bias(ba, M, N, dt):
    top = 1 if M >= 2 ** 22 else 2
    dY, Z = whole(M, N, dt, -1, top, 1), whole(M, N, dt, -1, 2, 2)
    ws = torch.empty(ba.bias_act_grad_workspace_size(M, N), dtype=torch.uint8, device="cuda")
    db = torch.full((N,), 0.5, device="cuda")
    ba.bias_act_grad(dY, Z, None, db, "relu", workspace=ws)
    check(db, lambda s: torch.where(Z[s] > 0, dY[s], 0).double(), M, N)
    db.fill_(0.5)
    ba.bias_act_grad(dY, None, None, db, workspace=ws)
    check(db, lambda s: dY[s].double(), M, N)


# 16385 and more: the kernels of long rows
NORM = [(1, 1, F32), (1, 4096, BF16), (37, 100, F16), (70000, 8, F32), (5000, 130, BF16), (4097, 1000, F16), (2500, 2048, F32), (32768, 4096, BF16),
        (1200, 5000, BF16), (700, 16000, F32), (300, 33000, F16), (5000, 16385, BF16), (32767, 16384, F32), (2 ** 23 - 1, 128, BF16),
        (16383, 65536, BF16), (3, 357913939, BF16)]


@pytest.mark.parametrize("rows,N,dt", NORM)
def test_norm_weights(ba, rows, N, dt):
    # statistics of 0 and 1: xhat is X itself
    dY, X = whole(rows, N, dt, -1, 1, 3), whole(rows, N, dt, -1, 1, 4)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    ws = torch.empty(ba.layer_norm_grad_workspace_size(rows, N), dtype=torch.uint8, device="cuda")
    dg, db = torch.full((N,), 0.5, device="cuda"), torch.full((N,), 0.5, device="cuda")
    ba.layer_norm_grad(dY, X, None, mean, rstd, torch.empty_like(X), dg, db, workspace=ws)
    check(dg, lambda s: dY[s].double() * X[s].double(), rows, N)
    check(db, lambda s: dY[s].double(), rows, N)
