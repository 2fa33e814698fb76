"""The quantising append keeps the sign of a zero, as e4m3(x / scale) does."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("peak", [3.0, 448.0, 2.0 ** -70, 2.0 ** 90, 0.0])
def test_negative_zero(cuda_lib, peak):
    """Rows with zeros of both signs beside a largest value whose scale is within and outside the range of
    the fast division, and a row of zeros alone."""
    g = torch.Generator().manual_seed(1)
    x = torch.zeros((6, 576), dtype=torch.bfloat16)
    x[:, :512] = torch.where(torch.rand((6, 512), generator=g) < 0.5, -0.0, 0.0)
    if peak:
        x[:, 17], x[3:, 300] = -peak, peak / 2
        x[4, 2] = -peak * 2.0 ** -30                   # rounds to zero: -0
    lat = torch.full((6, 512), 0x55, dtype=torch.uint8, device="cuda")
    scale, rope = torch.ones(6, device="cuda"), torch.zeros((6, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    cuda_lib.kv_append_quant(lat, scale, rope, slots, x.cuda())
    f = x[:, :512].float()
    s = f.abs().amax(1) / torch.full((6,), 448.0)
    ratio = f / s[:, None] if peak else f
    want = ratio.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(scale.cpu(), s)
    assert torch.equal(lat.cpu(), want)
    assert bool((want == 0x80).any()) and bool((want == 0).any())
    back = cuda_lib.kv_read_fp8(lat, scale, rope, slots).cpu()[:, :512]
    assert torch.equal(torch.signbit(back), torch.signbit(x[:, :512]))
