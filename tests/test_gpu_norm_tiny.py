"""Normed heads whose squares, and eps, are near or below float32's smallest numbers,
against float64, within the tolerances of test_gpu_norm_rope."""

import numpy as np
import pytest
import torch

from tests.test_gpu_norm_rope import BF16, F32, run_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,R", [(64, 32), (80, 20), (128, 128)])
@pytest.mark.parametrize("eps", [float(np.finfo(np.float32).tiny), 1e-40, 2e-45, 7e-31, 1e-29])
@pytest.mark.parametrize("size", [1e-14, 1e-18, 3e-20, 1e-22])
def test_tiny_eps(size, eps, D, R, dtype):
    """(eps as float32 holds it)"""
    run_case(30, 4, 2, D, R, 1, False, dtype, dtype, 16, 99, eps=float(np.float32(eps)), size=size,
             seed=12)
