"""The dS scratch of the cross-attention backward: sizes that ask for the
device's free memory, in a capture too."""
import pytest
import torch

from context_attention_long_b200 import api, build

from test_gpu_cross import lens_of, normal

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
