"""GPU residual norms: workgroups that walk down several rows at every width."""

import pytest
import torch

from gpu_support import need_gpu
from test_gpu_norm import test_forward_and_backward as forward_and_backward

pytestmark = pytest.mark.gpu


# B, S, D, post, gate, type of the parameters, quantized: workgroups of 2 or 3 rows forward and 2 to 6 backward, gate
# segments that end inside them, whole segments per workgroup and segments over several
@pytest.mark.parametrize("case", [(433, 3, 4096, 1, 1, torch.float32, ""), (100, 13, 5120, 1, 1, torch.bfloat16, "rows"),
                                  (1, 1300, 5120, 0, 1, torch.float32, ""), (550, 2, 8192, 1, 1, torch.float32, ""),
                                  (1, 1030, 8192, None, 0, torch.bfloat16, "rows"), (60, 10, 16384, 1, 1, torch.float32, ""),
                                  (300, 2, 10240, 1, 1, torch.bfloat16, "")], ids=str)
def test_workgroups_of_several_rows(case):
    need_gpu()
    forward_and_backward(case)
