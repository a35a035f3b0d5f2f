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


@pytest.mark.parametrize("ends", [(-3, 50), (0, 21), (-2 ** 31, 2 ** 31 - 1), (-1, 20)])
def test_q_start_is_clamped_as_in_the_attention(ends):
    """Tokens that are not there count neither in n_b nor in a token's place, so the attention finds what is appended."""
    s = case(2, 1, 64, 16, W.FP16, [5, 40], [7, 13], 32, 1, seed=41)
    s["q_start"] = np.array([ends[0], 7, ends[1]], np.int64).astype(np.int32)
    before = s["pool"].clone()
    out = call(s, False)
    s["q_start"] = np.clip(s["q_start"], 0, 20)
    assert check(s, out, before, False) == 0
