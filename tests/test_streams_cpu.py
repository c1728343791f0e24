"""What the binding allocates and clears for a call on a given stream belongs
to that stream (on the host, with stand-ins for the GPU and the library)."""
import contextlib

import pytest
import torch

import nvfp4_quantized_dense_amd as nv


class OnGpu(torch.Tensor):
    is_cuda = True


def t(*shape, dtype=torch.bfloat16):
    return torch.full(shape, 0, dtype=dtype).as_subclass(OnGpu)


class Calls:
    """The library: sizes as they are, every other call recorded and done."""

    def __init__(self, real):
        self.real, self.made = real, []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)
        return lambda *a: self.made.append(name) or nv.NVFP4_OK


@pytest.fixture
def log(monkeypatch):
    """(event, stream at hand) of all allocations, fills and stream changes; the library's calls in .calls."""
    events, now = [], []

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    def watch(owner, name):
        f = getattr(owner, name)
        monkeypatch.setattr(owner, name, lambda *a, **k: events.append((name, now[-1] if now else None)) or f(*a, **k))

    calls = Calls(nv.lib())
    monkeypatch.setattr(nv, "lib", lambda: calls)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda n: ("stream", n))
    for name in ("empty", "zeros"):
        watch(torch, name)
    watch(torch.Tensor, "zero_")
    events.clear()
    return events, calls


def attention(stream):
    cache = t(2, 2, 1, 18 * 64, dtype=torch.uint8)
    g = t(1, dtype=torch.float32)
    i32 = dict(dtype=torch.int32)
    nv.nvfp4_kv_attention(t(2, 4, 64), cache, t(2, 2, **i32), t(2, **i32), g, g, out=t(2, 4, 64), stream=stream)


def mlp(stream):
    w, g = t(16, dtype=torch.uint8), t(1, dtype=torch.float32)
    nv.mlp_forward(nv.MODE_W4A4, t(4, 256), w, g, w, g, 512, g, g, out=t(4, 256), stream=stream)


def mlp_awq(stream):
    w, g = t(16, dtype=torch.uint8), t(1, dtype=torch.float32)
    nv.mlp_forward_w4a16_awq(t(4, 256), w, g, t(256), w, g, t(512), 512, out=t(4, 256), stream=stream)


def silu(stream):
    nv.silu_mul_nvfp4_quant(t(2, 4, 64), t(2, dtype=torch.float32), stream=stream)


@pytest.mark.parametrize("call", [attention, mlp, mlp_awq, silu])
def test_workspaces_and_fills_are_on_the_calls_stream(call, log):
    events, calls = log
    call(777)
    assert len(calls.made) == 1
    made = [e for e in events if e[0] == ("zero_" if call is silu else "zeros" if call in (mlp, mlp_awq) else "empty")]
    assert made and all(s == ("stream", 777) for _, s in made)
    assert all(s == ("stream", 777) for e, s in events if e in ("zero_", "zeros"))  # no fill anywhere else
    events.clear()
    call(None)
    assert events and all(s is None for _, s in events)
