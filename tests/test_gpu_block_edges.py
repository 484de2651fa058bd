"""The block operators where rows, buffers, threads and limits meet their
edges. Comparisons and tolerances are those of test_gpu_blocks.py."""
import pytest
import torch

import matrix_aware_optimizer_gb300 as prm
from matrix_aware_optimizer_gb300 import native as N

from .gpu_helpers import ensure_built
from .test_gpu_blocks import BF16, FP16, FP32, _check_norm, _norm_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()
    N.load()
    yield
    prm.blocks_sync_status()


# ------------------------------------------- rows narrower than one 16-byte copy
@pytest.mark.parametrize("st,bt", [(FP32, FP32), (FP32, BF16), (BF16, BF16), (FP16, FP16)])
@pytest.mark.parametrize("d", [3, 5, 6, 7])
@pytest.mark.parametrize("B,L", [(2, 1), (5, 1), (6, 1), (7, 1), (10, 1), (14, 1), (40, 1), (9, 2)])
def test_norm_gradient_of_narrow_rows(B, L, d, st, bt):
    """A sample's rows are copied by themselves. Several samples at the end of
    a narrow tensor lie behind its last whole 16 bytes."""
    _check_norm(*_norm_case(B, L, d, "rms", st, bt, 1, 1, 1, 1, eps=1e-3))
    _check_norm(*_norm_case(B, L, d, "rms", st, bt, 0, 0, 0, 1, eps=1e-3))


@pytest.mark.parametrize("d,rows", [(3, 304 * 129 - 1), (3, 304 * 129 - 3), (5, 304 * 129 - 2), (7, 304 * 129)])
def test_norm_gradient_of_narrow_rows_without_samples(d, rows):
    """As many rows as leave one behind the last full step of 128 rows."""
    _check_norm(*_norm_case(1, rows, d, "rms", BF16, BF16, 1, 0, 1, 0, eps=1e-3))
