"""The norm and its gradients at widths that are no multiple of 8 and take two or
four chunks a lane, under the bounds of the other widths."""
import pytest

import test_gpu_ops as ops
from test_gpu_ops import gpu, named  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

# 1 chunk a lane up to 8192 (2048 forward, for many rows), 2 up to 16384, then 4.
WIDTHS = [4097, 8191, 8200, 9001, 16383, 16391, 20000, 32761, 32767]


@pytest.mark.parametrize("quantize", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("D", WIDTHS)
def test_rms_norm(D, residual, quantize):
    ops.test_rms_norm(D, residual, quantize)


@pytest.mark.parametrize("dres", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("D", WIDTHS)
def test_rms_norm_backward(D, dres):
    ops.test_rms_norm_backward(D, dres)
