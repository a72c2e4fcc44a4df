"""The forward's row maximum with every score far from zero: a maximum that takes
in anything but the row's own visible scores underflows the whole row."""
import numpy as np
import pytest
import torch

import joint_text_image_b200 as jt
from oracle import cache as oc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("level", [-300.0, 300.0])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_far_from_zero(level, D):
    S, Hq, Hkv = 200, 4, 2
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(1, S, h, D, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    q = (q.float() * 0.125).to(torch.bfloat16)
    q[..., 0] = 32.0
    k[..., 0] = float(round(level * D ** 0.5 / 32.0))
    seg = jt.hia_segments_build([(S, 0, 0, 0)], S)
    one, zero = torch.ones(1, S, D, device="cuda"), torch.zeros(1, S, D, device="cuda")
    o, lse = jt.hia_attn_fwd(seg, q.cuda(), k.cuda(), v.cuda(), one, zero)
    f64 = lambda t: t.double().cpu().numpy()
    ro, rl, ra = oc.attend(f64(q[0]), f64(k[0]), f64(v[0]), np.arange(S), D ** -0.5)
    # scores: one product of 32 * 107 beside D small ones (magnitudes <= 32 in
    # all): fp32 sums within 3460 * 2^-23 * sqrt(D) <= 4.7e-3, in an exponential
    # and the sum; weights and output rounded once each
    assert np.all(np.abs(f64(o[0]) - ro) <= 2.0 ** -8 * (ra + np.abs(ro)) * 1.01 + 1e-2 * ra)
    assert np.all(np.abs(f64(lse[0]) - rl) <= 5e-3)
