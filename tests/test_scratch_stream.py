"""The workspaces that the binding allocates by itself belong to the stream
that the call runs on: without a GPU, on stand-ins for the streams and for the
library, and (marked gpu) with the memory of a call in flight asked for again."""

import contextlib

import pytest
import torch

import gated_delta_net_causal_gb300 as gdn

BF = torch.bfloat16


class FakeLibrary:
    def __getattr__(self, name):
        return lambda *a: 0


@pytest.fixture
def allocations(monkeypatch):
    """The streams in force at each allocation of bytes; CPU tensors count as the current device's."""
    seen, current = [], ["current"]

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    real = torch.empty

    def empty(*a, **kw):
        if kw.get("dtype") == torch.uint8:
            seen.append(current[-1])
        return real(*a, **kw)

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(gdn, "library", FakeLibrary)
    monkeypatch.setattr(gdn, "_current_device", lambda: -1)
    monkeypatch.setattr(gdn, "_current_raw_stream", lambda dev: 0)
    for name in ("gdn_decay_prefill_workspace_size", "gdn_prefill_workspace_size", "gdn_decode_layer_workspace_size"):
        monkeypatch.setattr(gdn, name, lambda *a: 4096)
    return seen


def decay_prefill(stream):
    d, T = gdn.dims(1, 2, 64, io_dtype=BF), 5
    a = torch.zeros((T, 6 * 64), dtype=BF)
    gdn.gdn_decay_prefill(d, torch.tensor([0, T], dtype=torch.int32), a[:, :64], a[:, 64:128], a[:, 128:256],
                          torch.zeros(2), torch.zeros((1, 2, 64, 64)), out=torch.zeros((T, 2, 64), dtype=BF),
                          stream=stream)


def prefill_chunked(stream):
    d, T = gdn.dims(1, 2, 64, io_dtype=BF), 5
    z = lambda *s: torch.zeros(s, dtype=BF)
    with pytest.raises(ValueError):  # goes as far as the first address
        gdn.gdn_prefill_chunked(d, torch.tensor([0, T], dtype=torch.int32), z(T, 64), z(T, 64), z(T, 128), z(T, 2),
                                z(T, 2), torch.zeros(2), torch.zeros(2), torch.zeros((1, 2, 64, 64)), out=z(T, 2, 64),
                                core_out=torch.zeros((T, 2, 64)), stream=stream)


def decode_layer(stream):
    d, hidden, B = gdn.dims(1, 2, 64, io_dtype=BF), 64, 2
    z = lambda *s: torch.zeros(s, dtype=BF)
    with pytest.raises(ValueError):
        gdn.gdn_decode_layer(d, z(B, hidden), z(448, hidden), z(hidden, 128), z(256, 4), torch.zeros(2), torch.zeros(2),
                             torch.zeros(64), z(B, 256, 3), torch.zeros((B, 2, 64, 64)), z(B, hidden), stream=stream)


@pytest.mark.parametrize("call", [decay_prefill, prefill_chunked, decode_layer])
@pytest.mark.parametrize("stream,where", [(None, "current"), (0x7f0010, ("external", 0x7f0010)), (0, "default"),
                                          (1, "default")])
def test_allocated_on_the_stream_of_the_call(allocations, call, stream, where):
    call(stream)
    assert allocations == [where]


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [True, False])
def test_memory_of_a_call_in_flight_is_not_given_away(raw):
    """The call waits on a side stream while the current one allocates blocks of the workspace's size and fills them;
    and a block that queued work of the current stream still writes is not taken for a call on the other."""
    T, hk, hv, D = 1500, 1, 2, 128
    gen = torch.Generator().manual_seed(51)
    act = torch.randn((T, (2 * hk + hv) * D), generator=gen).to(BF).cuda()
    q, k, v = act.split([hk * D, hk * D, hv * D], dim=1)
    g = (-torch.rand(hv, generator=gen) * 0.01).cuda()
    S0 = torch.randn((1, hv, D, D), generator=gen).cuda()
    d, cu = gdn.dims(hk, hv, D, io_dtype=BF), torch.tensor([0, T], dtype=torch.int32, device="cuda")
    need = gdn.gdn_decay_prefill_workspace_size(d, 1, T)
    assert need > 0
    want, want_out = S0.clone(), torch.empty((T, hv, D), dtype=BF, device="cuda")
    gdn.gdn_decay_prefill(d, cu, q, k, v, g, want, out=want_out)
    S, out = S0.clone(), torch.empty_like(want_out)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    before = torch.empty(need, dtype=torch.uint8, device="cuda").fill_(0xff)  # written after the sleep
    del before
    with torch.cuda.stream(s):
        torch.cuda._sleep(40_000_000)
    gdn.gdn_decay_prefill(d, cu, q, k, v, g, S, out=out, stream=s.cuda_stream if raw else s)
    after = [torch.empty(need, dtype=torch.uint8, device="cuda").fill_(0xff) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(S, want) and torch.equal(out, want_out) and after
