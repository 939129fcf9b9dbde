"""Positions outside the rotation table where only part of a head is rotated,
against the float64 definition with the tolerances of test_gpu_norm_rope.
"""
import numpy as np
import pytest
import torch

from context_attention_long_b200 import api, build
from oracle import norm_rope as nr

from gpu_util import f64_of
from test_gpu_norm_rope import BF16, F32, _check_forward as check_forward, _inputs as inputs, _normal as normal, \
    _np as np_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


@pytest.mark.parametrize("S,H,Hk,D", [(9, 3, 2, 64), (9, 24, 8, 128), (4001, 2, 1, 128), (6001, 1, 1, 64)])
@pytest.mark.parametrize("interleaved", [True, False])
def test_positions_outside_the_table_with_part_of_a_head_rotated(S, H, Hk, D, interleaved):
    """The whole row is NaN, the elements behind the rotated part too, in both
    directions; other rows are right; the weight gradients, sums over all rows,
    are NaN in every column."""
    q, k, wq, wk, cos, sin, pos = inputs(1, S, H, Hk, D, D // 2, True, "f32", seed=12)
    pos[0, 3], pos[0, 5] = cos.shape[0], -1
    kw = dict(interleaved=interleaved)
    bad = torch.zeros(S, dtype=torch.bool, device="cuda")
    bad[3] = bad[5] = True
    outs = api.cpattn_qk_norm_rope(q, k, wq, wk, cos, sin, pos, **kw)
    assert api.cpattn_device_status() == (7, 1 << 7)
    gq, gk = normal(1, S, H, D, seed=8), normal(1, S, Hk, D, seed=9)
    dq, dk, dwq, dwk = api.cpattn_qk_norm_rope_backward(q, k, gq, gk, wq, wk, cos, sin, pos, **kw)
    assert api.cpattn_device_status() == (7, 1 << 7)
    for t in (*outs, dq, dk):
        assert bool(t[:, bad].isnan().all())
    assert bool(dwq.isnan().all()) and bool(dwk.isnan().all())
    keep = torch.arange(S, device="cuda")[~bad][:40]
    for x, y, w, g, dx in ((q, outs[0], wq, gq, dq), (k, outs[1], wk, gk, dk)):
        check_forward(x[:, keep], y[:, keep], w, cos, sin, pos[:, keep], **kw)
        # (a kept row's dx does not depend on the others; its weight gradient does)
        ref, _, size, _ = nr.norm_rope_backward(np_of(x[:, keep]), np_of(g[:, keep]), np_of(w), np_of(cos), np_of(sin),
                                                pos[:, keep].cpu().numpy(), **kw)
        assert np.all(np.abs(f64_of(dx[:, keep]) - ref) <= BF16 * np.abs(ref) + F32 * size)
