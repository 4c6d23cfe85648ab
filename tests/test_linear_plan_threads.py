"""The threads of a workgroup that gemm_linear_plan_cus states, for every kind of kernel."""
import pytest

from pipelined_tiled_dense_amd import binding as bd

# (M, N, K) with the tile that the plan has to have for the case to be one.
CASES = [("linear", 1, 4096, 8192, 16, 512), ("linear", 2048, 2048, 2048, 128, 512), ("linear", 4200, 4096, 136, 192, 512),
         ("linear", 8192, 8192, 8192, 256, 512), ("linear_bwd_weight", 32768, 1024, 1024, 256, 512),
         ("gated_linear", 37, 5005, 2048, 64, 512), ("gated_linear", 549, 2152, 544, 128, 256),
         ("gated_linear", 1936, 1024, 1216, 128, 256), ("gated_linear", 8192, 8192, 4096, 256, 512),
         ("gated_linear_bwd_input", 1936, 1024, 1216, 128, 512)]


@pytest.mark.parametrize("product,M,N,K,rows,threads", CASES)
def test_threads(product, M, N, K, rows, threads):
    p = bd.gemm_linear_plan_cus(M, N, K, product, 1, 1, 256)
    assert p["rows"] == rows and p["threads"] == threads
