"""What a kept few-token layer does on the host around its call (no GPU: the
call into the library is replaced, the buffers are host tensors)."""
import pytest

from sparse_mixture_experts_20_amd import binding as B


@pytest.fixture
def host(monkeypatch):
    """A namespace whose ``stream`` is the current stream's handle; ``used``
    lists the buffers whose use on another stream was recorded."""
    import torch

    class Host:
        stream = 0
        used = []
    h = Host()
    h.used = []
    monkeypatch.setattr(B, "_device_of", lambda t: t.get_device())
    monkeypatch.setattr(B, "_stream_of", lambda index: h.stream)
    monkeypatch.setattr(B, "_run", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: "stream")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: h.used.append(t.data_ptr()))
    return h


def _layer(**kw):
    import torch
    bf = torch.bfloat16
    w = (torch.zeros(4, 16), torch.zeros(4, 24, 16, dtype=bf), torch.zeros(4, 16, 24, dtype=bf))
    return w, B.FewLayer(*w, 2, 1.0, export=True, router_stats=True, **kw)


@pytest.mark.parametrize("home", [0, 4096])
def test_buffers_are_recorded_on_other_streams_only(host, home):
    import torch
    host.stream = home
    _, layer = _layer()
    x = torch.zeros(3, 16, dtype=torch.bfloat16)
    for _ in range(3):
        layer(x)
    assert host.used == []
    host.stream = 8192
    layer(x)
    buffers = [layer.workspace, *layer._routing, *layer._counts]
    assert sorted(host.used) == sorted(b.data_ptr() for b in buffers) and len(buffers) == 8
    host.used.clear()
    host.stream = home
    layer(x)
    assert host.used == []


def test_weights_stay_when_a_tensor_is_given_other_memory(host):
    import torch
    w, layer = _layer(act="gelu", b_up=torch.zeros(4, 24), b_down=torch.zeros(4, 16))
    held = [t.data_ptr() for t in layer.tensors]
    assert held[:3] == [t.data_ptr() for t in w]
    for t in w:
        t.data = torch.ones_like(t)
    assert [t.data_ptr() for t in layer.tensors] == held
    # what the descriptors hold: the pointer is a moe_tensor's first field
    assert [int.from_bytes(d[:8], "little") for d in layer._w] == held[:3]
    assert not any(bool(t.any()) for t in layer.tensors)
