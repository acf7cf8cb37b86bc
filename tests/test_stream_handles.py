"""Streams given to the dense operators as plain handles: 0 is the default stream, any other the stream itself."""
import contextlib

import pytest
import torch

from block_sparse_attention_41_b200 import sol_attn as sa


class FakeStream:
    def __init__(self, handle, device):
        self.cuda_stream, self.device = handle, device


def test_handle_zero_is_the_default_stream(monkeypatch):
    """On the CPU, with torch's stream classes replaced: its ExternalStream of handle 0 is a new stream of the pool,
    which does not wait for the default one."""
    entered = []

    def external(handle, device=None):
        return FakeStream(handle if handle else 0xbeef, device)

    @contextlib.contextmanager
    def stream(s):
        entered.append(s.cuda_stream)
        yield
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: FakeStream(0, device))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    for handle in (0, 0x1234):
        with sa._On(torch.device("cuda", 0), handle):
            pass
    assert entered == [0, 0x1234]


@pytest.mark.gpu
def test_a_call_on_handle_zero_follows_the_default_stream():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_attention_41_b200 import build
    build.build()
    with sa._On(torch.device("cuda", 0), 0):
        assert torch.cuda.current_stream().cuda_stream == 0
    g = torch.Generator(device="cuda").manual_seed(1)
    new = torch.randn((1, 600, 256), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn((256, 256), generator=g, device="cuda").to(torch.bfloat16)
    freq, _ = sa.sol_attn_rope_inv_freq(256, device="cuda")
    pos = torch.arange(600, dtype=torch.int32, device="cuda")
    calls = {"norm": lambda x, **k: sa.sol_attn_residual_norm(x, **k)[1],
             "norm gradient": lambda x, **k: sa.sol_attn_residual_norm_bwd(x, new, **k)["dx"],
             "rotary": lambda x, **k: sa.sol_attn_rope(x[None], None, pos, freq, **k)[0],
             "linear": lambda x, **k: sa.sol_attn_linear(x, w, **k),
             "linear gradient": lambda x, **k: sa.sol_attn_linear_bwd(x, new, w, **k)[0]}
    for name, call in calls.items():
        want = call(new)
        x = torch.zeros_like(new)
        torch.cuda.synchronize()
        torch.cuda._sleep(50_000_000)  # about 30 ms of the default stream before the input is there
        x.copy_(new)
        got = call(x, stream=0)
        torch.cuda.synchronize()
        assert torch.equal(got, want), name
