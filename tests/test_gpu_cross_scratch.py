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
    """302 MB of dS, which torch does not hold: the binding asks for the device's
    free memory, which a capture allows."""
    B, Sq, H, D, Skv = 1, 4608, 16, 64, 2048
    assert B * H * api.cpattn_cross_attention_backward_ds_bytes(H, H, Sq, Skv) > api._CROSS_DS_UNASKED
    q, dout = normal(B, Sq, H, D, seed=1), normal(B, Sq, H, D, seed=4)
    k, v = normal(B, Skv, H, D, seed=2), normal(B, Skv, H, D, seed=3)
    out, lse = api.cpattn_cross_attention(q, k, v)
    want = api.cpattn_cross_attention_backward(q, k, v, out, lse, dout)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
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


@pytest.mark.parametrize("B,Sq,H,Hk,D,Skv,lens,ranges", [
    (1, 4100, 8, 1, 64, 4200, None, 2),
    (1, 2300, 16, 1, 128, 4200, [4099], 2),
    (2, 5000, 21, 3, 64, 6000, [6000, 129], 2),        # groups of seven, an element of few tiles
    (2, 2400, 64, 2, 64, 4300, [0, 4300], 3),
    (2, 1024, 8, 1, 64, 40000, [40000, 129], 3),       # a run covers whole tiles, and more runs than steps
    (1, 1024, 8, 1, 128, 40000, None, 3),
    (1, 16384, 8, 1, 64, 16640, None, 17),
])
def test_a_pair_in_ranges_of_its_queries(B, Sq, H, Hk, D, Skv, lens, ranges):
    """The least workspace, which holds 256 MB of a pair's dS: dQ has the bytes
    of whole pairs, dK and dV, which add the same terms in another order, differ
    by their last rounding, and all of them are the same every run."""
    pair = api.cpattn_cross_attention_backward_ds_bytes(H, Hk, Sq, Skv)
    steps, q_tiles = (256 << 20) // ((Skv + 127) // 128 * 32768), (Sq + 127) // 128
    assert -(-(H // Hk * q_tiles) // steps) == ranges
    sizes = [api.cross_backward_workspace_bytes(B, H, Hk, Sq, Skv, D, ds_budget=n) for n in (0, 256 << 20, pair - 1, pair)]
    assert sizes[0] == sizes[1] == sizes[2] - (pair - 1) + (256 << 20) == sizes[3] - pair + (256 << 20)
    q, dout = normal(B, Sq, H, D, seed=1), normal(B, Sq, H, D, seed=4)
    k, v = normal(B, Skv, Hk, D, seed=2), normal(B, Skv, Hk, D, seed=3)
    n = lens_of(lens)
    out, lse = api.cpattn_cross_attention(q, k, v, n)
    args = (q, k, v, out, lse, dout, n)
    whole = api.cpattn_cross_attention_backward(*args)
    got = api.cpattn_cross_attention_backward(*args, ds_budget=0)
    again = api.cpattn_cross_attention_backward(*args, ds_budget=0)
    most = api.cpattn_cross_attention_backward(*args, ds_budget=pair - 1)     # all steps but one, then one
    assert torch.equal(got[0], whole[0]) and torch.equal(most[0], whole[0])
    for a, b, c, d in zip(got, again, most, whole):
        assert torch.equal(a, b)
        d = d.float()
        for t in (a, c):     # a step of bf16, and float32's 2^-24 of the magnitudes where they cancel
            assert bool(((t.float() - d).abs() <= 2.0 ** -7 * d.abs() + 2.0 ** -14 * d.abs().max()).all())
    if Sq * Skv * H * B < 1 << 28:
        check_norms(q, k, v, dout, [Skv] * B if lens is None else lens, got)
    assert api.cpattn_device_status() == (0, 0)
