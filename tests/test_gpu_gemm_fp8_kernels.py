"""Every kernel of the 8-bit product, in every form, on whole numbers and scales
that are powers of two: each partial sum fits fp32 and the fast way's grid, so the
result is the exact one, rounded, to the last bit.  test_gemm_fp8_plan.py checks
that the sizes reach the kernels."""
import pytest
import torch

import ops_reference as ref
from gemm_fp8_cases import CASES
from pipelined_tiled_dense_amd import binding as bd

pytestmark = pytest.mark.gpu

BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    bd.library()
    yield


@pytest.fixture(autouse=True)
def named(request):
    print("  %s" % request.node.name, flush=True)
    yield
    torch.cuda.synchronize()


def whole(g, rows, K, aligned):
    """Values -4 .. 4; rows on 16-byte boundaries or 3 bytes past them, K + 3 apart
    at least, with NaN bytes around."""
    ld, shift = (-(-K // 16) * 16, 0) if aligned else (K + 3 + (K % 16 == 13), 3)
    buf = torch.full((rows * ld + shift,), 0x7F, dtype=torch.uint8, device="cuda")
    q = buf[shift:].view(rows, ld)[:, :K]
    q.copy_(torch.randint(-4, 5, (rows, K), generator=g, device="cuda").float().to(FP8).view(torch.uint8))
    return q.view(FP8)


@pytest.mark.parametrize("case,want", CASES, ids=lambda v: "-".join(str(int(x)) for x in v))
def test_exact_result(case, want):
    M, N, K, b_rows, exact, a_aligned, b_aligned = case
    g = torch.Generator(device="cuda").manual_seed(M + 3 * N + 5 * K)
    a, b = whole(g, M, K, a_aligned), whole(g, N, K, b_aligned)
    power = lambda *s: 2.0 ** torch.randint(-1, 2, s, generator=g, device="cuda").float()  # noqa: E731
    sa, sb = power(ref.nblocks(K), M), power(ref.nblocks(K), -(-N // b_rows))
    full, _ = ref.gemm(a, sa, b, sb, b_rows)
    full = full.float()
    buf = torch.full((M + 1, N + 3), 7.0, dtype=BF16, device="cuda")
    for _ in range(2):     # the second time in kept memory
        assert torch.equal(bd.gemm_fp8(a, sa, b, sb, exact=exact, out=buf[:M, 1:N + 1]), full.to(BF16))
        assert (buf[M] == 7.0).all() and (buf[:, 0] == 7.0).all() and (buf[:, N + 1:] == 7.0).all()
    if exact:
        assert torch.equal(bd.gemm_fp8(a, sa, b, sb, out_dtype=torch.float32), full)
