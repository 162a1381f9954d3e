"""forward_routed on another stream than the current one: the memory that it
drops at its end must not be handed out on the current stream while the other
still uses it, and the result is the same."""
import pytest
import torch

import moe_synth
from top_routed_expert_gb300 import abi
from top_routed_expert_gb300.layer import MoELayer

pytestmark = pytest.mark.gpu


def test_memory_stays_with_the_stream(monkeypatch):
    T, E, k, d = 64, 32, 4, 256
    moe = MoELayer(moe_synth.make_custom(T=T, d=d, E=E, k=k, f=128, fs=128, x_dtype="bf16", w_dtype="e4m3", seed=2))
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
    w = torch.full((T, k), 0.25, device="cuda")
    want = moe.forward_routed(x, ids, w)
    torch.cuda.synchronize()
    used = []
    permute, ffn = abi.moe_permute, abi.moe_expert_ffn

    def keep(call):
        def f(cfg, *a, **kw):
            used.extend((t.data_ptr(), t.numel() * t.element_size()) for t in a
                        if isinstance(t, torch.Tensor) and t.data_ptr() not in held)
            return call(cfg, *a, **kw)
        return f
    held = {t.data_ptr() for t in (x, ids, w, moe.workspace(T))}
    monkeypatch.setattr(abi, "moe_permute", keep(permute))
    monkeypatch.setattr(abi, "moe_expert_ffn", keep(ffn))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                     # the kernels come some milliseconds after the call
    y = moe.forward_routed(x, ids, w, stream=side)
    # not written: whose memory it is shows in its address
    new = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in used for _ in range(3)]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in new]
    assert used and not any(a < q and p < a + n for a, n in used for p, q in spans)
    side.synchronize()
    assert abi.moe_get_device_status() == 0 and torch.equal(y, want)
