"""Time-outs in the 8-bit block's calls are reported by its check, whichever call they happened in.

A wait that runs out is made by the library's probe on the very workspace that the call's kernels report to."""
import pytest
import torch

from test_gpu_fp8_layer import make_block, tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    from serve_invariant_moe_gb300 import build
    build.build()


def reported(obj):
    from serve_invariant_moe_gb300._lib import InvmoeError
    with pytest.raises(InvmoeError) as e:
        obj.check()
    obj.check()
    return e.value.code == -6


def test_prefill_decode_and_graph():
    from serve_invariant_moe_gb300 import binding, block
    blk = make_block()
    x, res = tokens(40, blk.w.H, dtype=torch.bfloat16)
    want, _ = blk.prefill(x, res)
    blk.check()
    first = blk.prefill(x[:5].contiguous(), res[:5].contiguous(), return_all=True)["workspace"]
    binding.debug_timeout_probe(first, timeout_us=2000)
    blk.prefill(x.repeat(80, 1), res.repeat(80, 1))          # replaces the workspace
    assert reported(blk)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ws = blk.prefill(x, res, return_all=True)["workspace"]
        binding.debug_timeout_probe(ws, timeout_us=2000)
    assert reported(blk)
    blk.decode(x[:2].contiguous(), res[:2].contiguous())
    binding.debug_timeout_probe(blk._bufs["ws"], timeout_us=2000)
    blk.decode(x, res)
    assert reported(blk)
    g = block.Fp8DecodeGraph(blk, 3)
    g.check()
    binding.debug_timeout_probe(g._bufs["ws"], timeout_us=2000)
    assert reported(g)
    # and everything still computes the same
    g.x.copy_(x[:3])
    g.residual.copy_(res[:3])
    assert torch.equal(g.replay()[0], want[:3]) and torch.equal(blk.prefill(x, res)[0], want)
    blk.check()
    g.check()
