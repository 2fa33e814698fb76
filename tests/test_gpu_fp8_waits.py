"""The fp8 attention's bounded waits with many key tiles a CTA: every role is somewhere in its loop when
the wait on the first tile (withheld by the test hook) runs out."""
import numpy as np
import pytest
import torch

from counted_keys import Counted
from test_gpu_fp8_keys import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_len,H,lengths,nsplit", [(9, 8, [1500], 1), (10, 8, [1500], 1), (1, 96, [2000], 2),
                                                    (2, 4, [700, 60, 9000], 0), (1, 8, [60] * 70, 0)])
def test_expired_waits_end_the_call(cuda_lib, q_len, H, lengths, nsplit):
    """The status says so, the outputs are finite, and the next call on the same buffers is right."""
    mv = cuda_lib
    c = Counted(q_len, H, lengths, seed=1, mask=True)
    dev = lambda x: torch.from_numpy(x).cuda()
    q = torch.zeros((c.B, q_len, H, 576), dtype=torch.bfloat16, device="cuda")
    mv.device_status(clear=True)
    assert mv.load().mla_debug_stall_next_launch() == 0
    out, _ = mv.verify_attn_fp8(q, dev(c.lat), dev(c.scale), dev(c.rope).to(torch.bfloat16), dev(c.table), dev(c.seq),
                                dev(c.mask), 1.0, nsplit=nsplit)
    torch.cuda.synchronize()
    assert mv.device_status(clear=True) == mv.DEV_TIMEOUT
    assert bool(torch.isfinite(out).all())
    check(mv, c, nsplit=nsplit)
