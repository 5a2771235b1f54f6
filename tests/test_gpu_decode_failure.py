"""A decode whose prompts' kernel gives up: a key tile is never loaded, the bounded waits run out, and the join meets a
workspace in which no partial results of the prompt were written (it is filled with bytes of 0x7f, as counts and places
far outside it).  The call ends, the host reads the status, and the next calls are right."""
import time

import pytest
import torch

from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk
from test_gpu_decode import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which,bits", [(6, 16), (7, 4)])
def test_a_prompt_that_is_never_loaded(which, bits):
    pbuild.build()
    c = Case([0, 40], [7_001], [i % 50 for i in range(40)], 32, 8, 128, 64, bits, seed=90)
    want = c.run()
    dk.dualkv_check_status()
    t0 = time.time()
    dk.dualkv_selftest_kernel(which, 50_000_000)
    with pytest.raises(dk.DualKVError) as ei:
        dk.dualkv_check_status()
    assert ei.value.code == dk.DUALKV_ERR_DEVICE
    assert time.time() - t0 < 30
    dk.dualkv_check_status()  # the status word was cleared
    got = c.run()
    dk.dualkv_check_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.check(*got)
