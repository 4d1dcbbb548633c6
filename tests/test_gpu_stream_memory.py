"""The calls that run on a ``stream`` of their own make their outputs from that stream's memory: memory just freed on the current
stream may still be written by work that is queued there, which the other stream does not wait for."""
import pytest
import torch

import gated_delta_rule_looped_b200 as lt2
from tests.test_gpu_glr import backward, forward, make
from tests.test_gpu_kv_append import setup as append_setup
from tests.test_gpu_swa_decode import ALL, setup as attend_setup

pytestmark = pytest.mark.gpu


def calls():
    """name -> (a call that takes a stream, and returns all tensors that it makes)"""
    v = make(2, 4, 8, 700, 128, "bf16", "bf16", True, True, True, 1)
    one = make(2, 64, 16, 1, 128, "bf16", "bf16", True, True, True, 2)
    x, a, b = (one[n][:, :, :, 0].contiguous() for n in ("x", "a", "b"))
    a_s = append_setup(2, 8, 4, 128, 64, [4, 400, 77], [70, 190, 300], "bf16", 3)
    d = attend_setup(2, 64, 4, 128, 64, [1100, 1090, 1300] * 8, ALL, "bf16", 4, prefix=1024)
    rope = lt2.make_rope(128)
    return {
        "prefill": lambda **kw: forward(v, save_states=True, **kw),
        "backward": lambda **kw: [t for t in backward(v, **kw).values()],
        "decode": lambda **kw: [lt2.glr_decode(x, a, b, one["S0"], S_out=torch.empty_like(one["S0"]), gate_logits=True, **kw)],
        "append": lambda **kw: lt2.kv_append(a_s["q"], a_s["k"], a_s["v"], a_s["kc"], a_s["vc"], a_s["table"], a_s["start"],
                                             cu_seqlens=a_s["cu"], rope=rope, k_out=True, **kw),
        "attend": lambda **kw: [lt2.swa_decode(d["q"], d["kc"], d["vc"], d["table"], d["n"], prefix_len=1024, **kw)],
    }


@pytest.mark.parametrize("name", ["prefill", "backward", "decode", "append", "attend"])
@pytest.mark.parametrize("handle", [False, True])
def test_outputs_do_not_take_memory_freed_on_the_current_stream(name, handle):
    call = calls()[name]
    ref = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    # blocks of the outputs' sizes, freed on the current stream: the first that its next tensors would take
    freed = [torch.empty_like(t) for t in ref]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in freed]
    del freed
    got = call(stream=s.cuda_stream if handle else s)
    for t in got:
        assert all(t.data_ptr() + t.numel() * t.element_size() <= lo or t.data_ptr() >= hi for lo, hi in spans)
    torch.cuda.current_stream().wait_stream(s)
    assert name == "append" or all(torch.equal(a, b) for a, b in zip(got, ref))
    torch.cuda.synchronize()
    assert lt2.lt2_gdr_last_device_error() == lt2.LT2_OK
    # while another stream is current, the call's own stream counts as before
    with torch.cuda.stream(s):
        again = call()
    torch.cuda.synchronize()
    assert name == "append" or all(torch.equal(a, b) for a, b in zip(again, ref))
