"""A call given the default stream by its handle, 0, while another stream is
current: its outputs are the default stream's memory, as torch's allocator
lists it, and hold the same bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp4_block_scaled_quantize_amd")


def _owner(t):
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in torch's memory")


def test_outputs_of_handle_zero_are_the_default_streams():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator().manual_seed(1)
    z = torch.randn(3, 9000, generator=g).cuda()
    x, r, w = (torch.randn(*s, generator=g).cuda() for s in ((5, 264), (5, 264), (264,)))
    want = (fq.fp4_token_logprobs(z, top=3), *fq.fp4_residual_norm(x, r, w))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = (fq.fp4_token_logprobs(z, top=3, stream=0), *fq.fp4_residual_norm(x, r, w, stream=0))
        own = fq.fp4_residual_norm(x, r, w)
    torch.cuda.synchronize()
    for a, b in zip((got[0].entropy, got[0].top_ids, *got[1:]), (want[0].entropy, want[0].top_ids, *want[1:])):
        assert torch.equal(a, b) and _owner(a) == 0
    assert all(_owner(t) == side.cuda_stream for t in own)
