"""The plan of the attention of one token on the present device, and the forms of its splits that ordinary sizes take."""
import ctypes

import pytest
import torch

from tests.test_gpu_serve import kda  # noqa: F401
from tests.test_serve_plan import plan

pytestmark = pytest.mark.gpu


def test_the_device_is_asked(kda):  # noqa: F811
    """Without a given device the plan is for the present one's SMs; a whole GB300 places clusters of 16."""
    lib, sms = kda.load(), torch.cuda.get_device_properties(0).multi_processor_count
    lib.kda_debug_attend_plan.restype = ctypes.c_int
    for dtype in (0, 1):
        for K in (64, 128):
            for HQ, HKV in ((4, 4), (16, 4), (16, 2), (20, 2)):
                for N, rows in ((1, 900), (1, 2048), (2, 9000), (1, 65536), (64, 8192), (300, 40)):
                    assert plan(lib, HQ, HKV, K, K, dtype, N, rows, sms=0) == plan(lib, HQ, HKV, K, K, dtype, N, rows, sms=sms)
