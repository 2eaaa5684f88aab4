"""QLinear on another device than the current one is refused before the library is called (no GPU: tensors are
stand-ins that say where they are)."""
import pytest

from test_kv_binding import Library, Tensor

torch = pytest.importorskip("torch")


@pytest.fixture
def layer(qlin, monkeypatch):
    lib = Library()
    monkeypatch.setattr(qlin, "lib", lambda: lib)
    monkeypatch.setattr(qlin, "_stream", lambda s: s)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: Tensor(shape, dtype, int(str(device).split(":")[1])))
    q = object.__new__(qlin.QLinear)
    q.handle = type("Handle", (), {"ptr": None})()
    q.format, q.N, q.K, q.weights = qlin.FMT_W4G128, 256, 128, None
    return q, lib


def calls(q, X, Y):
    return {"qlin_forward": lambda: q(X), "qlin_forward ": lambda: q(X, out=Y), "qlin_act_quant": lambda: q.act_quant(X),
            "qlin_forward_acc": lambda: q.forward_acc(X), "qlin_forward_host": lambda: q.forward_host(X, Y, X, Y)}


@pytest.mark.parametrize("weights", [0, None])
def test_on_the_current_device(layer, weights):
    q, lib = layer
    q.weights = None if weights is None else Tensor((1000,), torch.uint8, weights)
    for name, call in calls(q, Tensor((2, 128), torch.bfloat16, 0), Tensor((2, 256), torch.bfloat16, 0)).items():
        call()
        assert lib.calls[-1] == name.strip()


@pytest.mark.parametrize("weights,x,y", [(1, 1, 1), (1, 0, 0), (0, 1, 0), (None, 1, 1)])
def test_elsewhere_is_refused(layer, weights, x, y):
    q, lib = layer
    q.weights = None if weights is None else Tensor((1000,), torch.uint8, weights)
    for call in calls(q, Tensor((2, 128), torch.bfloat16, x), Tensor((2, 256), torch.bfloat16, y)).values():
        with pytest.raises(ValueError, match="current device"):
            call()
    if weights:
        with pytest.raises(ValueError, match="current device"):
            q.dequant_device()
    assert lib.calls == []
