"""The outputs that the 8-bit block's calls allocate are tensors like torch's own: dispatch modes see them made, and the
deterministic fill of uninitialised memory reaches them."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _build():
    from serve_invariant_moe_gb300 import build
    build.build()


class Record(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.made = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        self.made.append((str(func), out))
        return out


def test_dispatch_modes_see_the_outputs():
    from serve_invariant_moe_gb300 import binding
    x, w = torch.randn(5, 256, device=DEV), torch.ones(256, dtype=torch.bfloat16, device=DEV)
    want = binding.add_rms_norm(x, w, fp8=True)
    with Record() as r:
        got = binding.add_rms_norm(x, w, fp8=True)
        routed = binding.moe_route_select(x, 2)
    made = [t.data_ptr() for name, t in r.made if "empty" in name]
    outputs = [got[n] for n in ("out", "q", "scale", "rstd")] + [routed["topk_idx"], routed["topk_w"]]
    assert made == [t.data_ptr() for t in outputs]
    for n in ("out", "scale", "rstd"):
        assert torch.equal(got[n], want[n])
    for t in outputs:
        like = torch.empty(t.shape, dtype=t.dtype, device=DEV)
        assert t.device == like.device and t.stride() == like.stride() and t.requires_grad == like.requires_grad


def test_the_deterministic_fill_reaches_new_outputs():
    from serve_invariant_moe_gb300 import binding
    x = torch.randn(5, 256, device=DEV)
    poison = torch.zeros(1 << 20, device=DEV)          # so that what the allocator hands out next is not NaN by chance
    del poison
    before = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)
    try:
        m = binding.marshal()
        for code, dtype in ((binding.BF16_, torch.bfloat16), (binding.F32_, torch.float32), (binding.I32_, torch.int32)):
            new, like = m.new(x, code, 7, 300), torch.empty(7, 300, dtype=dtype, device=DEV)
            assert new.dtype == dtype
            assert torch.isnan(new).all() if dtype.is_floating_point else torch.equal(new, like)
    finally:
        torch.use_deterministic_algorithms(before)
