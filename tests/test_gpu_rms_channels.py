"""Channel RMS norm over every count of 8-channel vectors per lane (1, 2, 3 and 4), through the C ABI.

768 channels are 3 vectors for each of 32 lanes; the sum of squares and the outputs must stay inside the pixel's
own channels, up to the last pixel.  fp32 in and out against the float64 oracle: at most 1e-5 of max|ref| (the
fp32 sum of C squares is off by at most C * 2^-24 of itself, its square root by half that: 3.1e-5 / 2 at
C = 1024 in the worst case and far less for a sum in 32 or more parts; the rest is a few roundings).
"""
import numpy as np
import pytest
import torch

from oracle import ops
from patch_tiled_causal_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Cc", [8, 64, 256, 512, 768, 1024])
def test_rmsnorm_stays_inside_its_channels(Cc):
    from patch_tiled_causal_gb300 import build, vaedec as vd
    build.build()
    B, T, H, W = 1, 2, 3, 5
    x = (synth.draw_normal((B, T, H, W, Cc), 3) * np.exp2(np.arange(W) - 2.0)[:, None]).astype(np.float32)
    gamma, beta = (1 + 0.2 * synth.draw_normal((Cc,), 4)).astype(np.float32), synth.draw_normal((Cc,), 5).astype(np.float32)
    n = x.size
    buf = torch.full((n + 4096,), -77.0, device="cuda")  # values behind the last pixel, in reach of a lane
    y = buf[:n].view(B, T, H, W, Cc)
    xb = torch.full((n + 4096,), 9.0, device="cuda")
    xb[:n] = torch.from_numpy(x).cuda().flatten()
    vd.channel_rmsnorm_silu(xb[:n].view(B, T, H, W, Cc), torch.from_numpy(gamma).cuda(), torch.from_numpy(beta).cuda(), y,
                            B, T, H, W, Cc, silu=True)
    ref = ops.silu(ops.channel_rms_norm(x.astype(np.float64).transpose(0, 4, 1, 2, 3), gamma, beta, 1e-6))
    ref = ref.transpose(0, 2, 3, 4, 1)
    got = y.cpu().numpy()
    assert np.abs(got - ref).max() <= 1e-5 * np.abs(ref).max()
    assert (buf[n:] == -77).all()
