"""Which stream the outputs and workspaces of a call belong to, seen from the
host: the one that the call's work is queued on, whatever form the caller
names it in.  Handle 0 is the default stream (what
torch.cuda.current_stream().cuda_stream gives a caller who has set nothing);
torch's ExternalStream(0) is not that stream but a new one."""
import contextlib
import subprocess
import sys

import pytest
import torch

import fp4_block_scaled_quantize_amd as fq
from tests.conftest import ROOT

BF = torch.bfloat16


class _Handle:
    def __init__(self, name):
        self.name = name


class _Library:
    """Every call succeeds; workspaces are asked for; the streams are kept."""
    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        if name.endswith("_workspace"):
            return lambda *a: 64

        def call(*a):
            self.streams.append(a[-1])
            return 0
        return call


@pytest.fixture
def host(monkeypatch):
    """CPU tensors stand in for the device's; `made` holds the stream current
    at each allocation."""
    lib, made, current = _Library(), [], ["caller's"]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream.name)
        yield
        current.pop()

    for name in ("empty", "empty_like"):
        real = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, _real=real, **k: (made.append(current[-1]), _real(*a, **k))[1])
    monkeypatch.setattr(fq, "lib", lambda: lib)
    monkeypatch.setattr(fq, "_on_device", lambda what, *t: torch.device("cpu"))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: _Handle("default"))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, device=None: _Handle(f"external {ptr}" if ptr else "a new one"))
    return lib, made


def _calls(stream):
    x, slots = torch.zeros(4, 256, dtype=BF), torch.zeros(4, dtype=torch.int32)
    bank = fq.LoraBank(torch.zeros(2, 16, 256, dtype=BF), torch.zeros(2, 64, 16, dtype=BF), torch.ones(2))
    w = fq.QTensor(torch.zeros(64, 128, dtype=torch.uint8), torch.zeros(64, 16, dtype=torch.uint8), torch.zeros(2), 64, 256, 16,
                   "e4m3")
    z, tok, wt = torch.zeros(4, 100), torch.zeros(4, dtype=torch.long), torch.ones(256)
    saved = fq.TokenLogprobs(torch.zeros(4), torch.zeros(4), torch.zeros(4, 2), None, None)
    return {
        "fp4_lora_apply": lambda: fq.fp4_lora_apply(x, bank, slots, stream=stream),
        "fp4_lora_backward": lambda: fq.fp4_lora_backward(torch.zeros(4, 64, dtype=BF), x, torch.zeros(4, 16), bank, slots,
                                                          stream=stream),
        "fp4_wo_gemm_lora": lambda: fq.fp4_wo_gemm_lora(x, w, bank, slots, stream=stream),
        "fp4_token_logprobs": lambda: fq.fp4_token_logprobs(z, tok, top=2, stream=stream),
        "fp4_token_logprobs_backward": lambda: fq.fp4_token_logprobs_backward(z, tok, saved, torch.ones(4), stream=stream),
        "fp4_residual_norm": lambda: fq.fp4_residual_norm(x, x, wt, stream=stream),
        "fp4_residual_norm_backward": lambda: fq.fp4_residual_norm_backward(x, x, x, x, wt, torch.zeros(4, 2), stream=stream),
    }


@pytest.mark.parametrize("name", list(_calls(0)))
@pytest.mark.parametrize("handle,owner", [(0, "default"), (4096, "external 4096")])
def test_memory_belongs_to_the_stream_of_the_handle(host, name, handle, owner):
    lib, made = host
    call = _calls(handle)[name]
    made.clear()
    call()
    assert lib.streams == [handle]
    assert made and set(made) == {owner}


def test_current_stream_without_torchs_private_call():
    """The calls of every operator ask for the current stream's handle; a torch
    that lacks the private function for it leaves the public one."""
    code = (
        "import torch\n"
        "if hasattr(torch._C, '_cuda_getCurrentRawStream'):\n"
        "    del torch._C._cuda_getCurrentRawStream\n"
        "import fp4_block_scaled_quantize_amd as fq\n"
        "class Stream:\n"
        "    def __init__(self, index): self.cuda_stream = 70 + index\n"
        "torch.cuda.current_stream, torch.cuda.current_device = Stream, lambda: 2\n"
        "assert fq._stream(None, torch.device('cuda', 3)) == 73 and fq._stream(None) == 72\n")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)
