"""The dS scratch of the cross-attention backward: sizes that ask for the
device's free memory, in a capture too; launches of some of the (batch element,
key head) pairs; offsets past 32 bits."""
import pytest
import torch

from context_attention_long_b200 import api, build

from test_gpu_cross import lens_of, normal
from test_gpu_cross_backward import check_backward
from test_gpu_cross_few_states import check_norms

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def test_large_scratch_in_a_capture():
    """302 MB of dS: the binding asks for the free memory, which a capture allows."""
    B, Sq, H, D, Skv = 1, 4608, 16, 64, 2048
    assert B * H * api.cpattn_cross_attention_backward_ds_bytes(H, H, Sq, Skv) > api._CROSS_DS_UNASKED
    q, dout = normal(B, Sq, H, D, seed=1), normal(B, Sq, H, D, seed=4)
    k, v = normal(B, Skv, H, D, seed=2), normal(B, Skv, H, D, seed=3)
    out, lse = api.cpattn_cross_attention(q, k, v)
    want = api.cpattn_cross_attention_backward(q, k, v, out, lse, dout)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = api.cpattn_cross_attention_backward(q, k, v, out, lse, dout)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("pairs", [1, 3, 4])
@pytest.mark.parametrize("lens", [None, [300, 0, 129], [5, 300, 200]])
def test_groups_of_pairs_that_end_inside_a_batch_element(pairs, lens):
    """Three elements of two key heads in launches of `pairs` pairs: dQ has the
    bytes of the launch for all, dK and dV, whose runs are cut elsewhere, are
    right."""
    B, Sq, H, Hk, D, Skv = 3, 150, 6, 2, 64, 300
    q, dout = normal(B, Sq, H, D, seed=1), normal(B, Sq, H, D, seed=4)
    k, v = normal(B, Skv, Hk, D, seed=2), normal(B, Skv, Hk, D, seed=3)
    n = lens_of(lens)
    out, lse = api.cpattn_cross_attention(q, k, v, n)
    pair = api.cpattn_cross_attention_backward_ds_bytes(H, Hk, Sq, Skv)
    want = api.cpattn_cross_attention_backward(q, k, v, out, lse, dout, n)
    got = api.cpattn_cross_attention_backward(q, k, v, out, lse, dout, n, ds_budget=pairs * pair)
    assert torch.equal(got[0], want[0])
    check_backward(q, k, v, dout, lens, got)
    check_norms(q, k, v, dout, [Skv] * B if lens is None else lens, got)


@pytest.mark.parametrize("Hk", [1, 2])
def test_scratch_past_4_gb(Hk):
    """4.4 GB of dS in one launch, of one pair or of two: dQ of the last head
    and of one in the middle has the bytes of that head alone."""
    Sq, H, D, Skv = 16384, 8, 64, 16640
    assert Hk * api.cpattn_cross_attention_backward_ds_bytes(H, Hk, Sq, Skv) > 1 << 32
    q, dout = normal(1, Sq, H, D, seed=1), normal(1, Sq, H, D, seed=4)
    k, v = normal(1, Skv, Hk, D, seed=2), normal(1, Skv, Hk, D, seed=3)
    out, lse = api.cpattn_cross_attention(q, k, v)
    dq = api.cpattn_cross_attention_backward(q, k, v, out, lse, dout, ds_budget=8 << 30)[0]
    for h in (3, 7):
        one = slice(h, h + 1)
        g = slice(h // (H // Hk), h // (H // Hk) + 1)
        alone = api.cpattn_cross_attention_backward(q[:, :, one], k[:, :, g], v[:, :, g], out[:, :, one].contiguous(),
                                                    lse[:, one].contiguous(), dout[:, :, one].contiguous())[0]
        assert torch.equal(dq[:, :, one], alone)
    assert api.cpattn_device_status() == (0, 0)
