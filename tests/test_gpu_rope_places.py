"""argus_rope_append: where tokens go when the table or q_start leave them little room."""

import numpy as np
import pytest
import torch

from mixed_precision_paged_argus_gb300 import workloads as W
from test_gpu_rope import DEV, call, case, check

pytestmark = pytest.mark.gpu


def test_an_empty_table_stores_nothing():
    s = case(2, 1, 64, 16, W.FP16, [0, 3], [9, 4], 32, 1, seed=40)
    s["table"], s["codec"], s["max_pages"] = np.zeros((2, 0), np.int32), np.zeros((2, 0), np.uint8), 0
    before = s["pool"].clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert check(s, call(s, False, status=status), before, False) == 13 and int(status) == 13
