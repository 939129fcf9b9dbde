"""Calls of the operators on a stream that is not the current one: what a call
allocates may share no block with work still queued on the current stream, and
what it returned may not be handed out while the current stream still reads it.

The current stream is kept busy by a long spin; blocks of the size that the
call is about to need are written and dropped behind it, so that an allocation
from the current stream's pool would get one of them.  Everything compared has
the bytes of the same call on the current stream.
"""
import pytest
import torch

from context_attention_long_b200 import api, build

from test_gpu_cross import lens_of, normal

pytestmark = pytest.mark.gpu
SPIN = 200_000_000      # clock cycles, some 0.1 s


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def _calls():
    """name -> (call(stream) returning its outputs, bytes of the blocks that it allocates)."""
    B, S, H, Hk, D, n = 2, 300, 4, 2, 64, 170
    q, k, v, g = normal(B, S, H, D, seed=1), normal(B, n, Hk, D, seed=2), normal(B, n, Hk, D, seed=3), normal(B, S, H, D, seed=4)
    lens = lens_of([170, 33])
    w = torch.linspace(0.5, 1.5, D, device="cuda")
    angle = torch.linspace(0, 3, S * D // 2, device="cuda").view(S, D // 2)
    cos, sin = angle.cos(), angle.sin()
    out, lse = api.cpattn_cross_attention(q, k, v, lens)
    ws = api.cross_backward_workspace_bytes(B, H, Hk, S, n, D)
    wsn = api.cpattn_qk_norm_rope_backward_workspace_bytes(D)
    qb, kb, lb = q.numel() * 2, k.numel() * 2, lse.numel() * 4
    kt = normal(B, S, Hk, D, seed=5)
    gk = normal(B, S, Hk, D, seed=6)
    return {
        "cross": (lambda s: api.cpattn_cross_attention(q, k, v, lens, stream=s), [qb, lb]),
        "cross one token": (lambda s: api.cpattn_cross_attention(q[:, :1], k, v, lens, stream=s), [B * H * D * 2, B * H * 4]),
        "cross backward": (lambda s: api.cpattn_cross_attention_backward(q, k, v, out, lse, g, lens, stream=s),
                           [qb, kb, kb, ws]),
        "norm": (lambda s: api.cpattn_qk_norm_rope(q, kt, w, w, cos, sin, stream=s), [qb, kt.numel() * 2]),
        "norm backward": (lambda s: api.cpattn_qk_norm_rope_backward(q, kt, g, gk, w, w, cos, sin, stream=s),
                          [qb, kt.numel() * 2, D * 4, D * 4, wsn]),
    }


NAMES = ["cross", "cross one token", "cross backward", "norm", "norm backward"]


@pytest.mark.parametrize("name", NAMES)
def test_allocations_share_no_block_with_the_current_stream(name):
    call, sizes = _calls()[name]
    want = [t.clone() for t in call(None)]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(SPIN)
    for _ in range(3):
        held = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
        for t in held:
            t.fill_(0xA5)                   # queued behind the spin
        del held, t
    got = call(stream)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert api.cpattn_device_status() == (0, 0)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_live_until_the_current_stream_has_read_them(name):
    call, _ = _calls()[name]
    want = [t.clone() for t in call(None)]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(stream)
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda._sleep(SPIN)
    copies = [t.clone() for t in got]       # queued behind the spin
    del got
    with torch.cuda.stream(stream):         # further allocations of that stream, written at once
        again = [torch.full_like(t, 7) for t in want]
    torch.cuda.synchronize()
    for a, b in zip(copies, want):
        assert torch.equal(a, b)
    del again
