"""The attention plans' calls beside other users of the device and the thread."""
import pytest
import torch

import chip_fusion_amd as cf

pytestmark = pytest.mark.gpu


def test_an_earlier_error_of_the_thread_is_not_the_calls():
    """An unrelated call has failed and nobody has asked for its error: the plans'
    calls are launched, once, and report none."""
    H, D, n = 2, 64, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((n, H, D), generator=g, device="cuda").half() for _ in range(3))
    s0, decay = torch.randn((n, H, D, D), generator=g, device="cuda"), torch.full((H,), -0.5, device="cuda")
    cu, O, O2 = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.empty_like(q), torch.empty_like(q)
    plan, att, L = cf.LinearAttention("f16", H, H, D), cf.Attention("f16", H, H, D), cf.lib()
    want, after = plan.step(q, k, v, decay, s0)
    want2 = att.run(q, k, v, cu)
    torch.cuda.synchronize()
    for stream in (None, torch.cuda.current_stream()):            # compiled and in Python
        s = s0.clone()
        torch.cuda.synchronize()
        print(f"\n[case] an earlier error, stream {stream}", flush=True)
        try:
            assert L.hipSetDevice(1 << 20) != 0                   # no such device: the host says so
            plan.step(q, k, v, decay, s, O=O, state_out=s, stream=stream)
            att.run(q, k, v, cu, O=O2, stream=stream)
        finally:
            L.hipGetLastError()
        torch.cuda.synchronize()
        assert torch.equal(O, want) and torch.equal(s, after) and torch.equal(O2, want2)
