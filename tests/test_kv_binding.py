"""The cache's Python binding without a GPU: what it refuses before the library is called.  Tensors are
stand-ins that say they are on a device."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")


class Tensor:
    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device, self._d, self.is_cuda = shape, dtype, f"cuda:{device}", device, True

    def get_device(self):
        return self._d

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def stride(self, i=None):
        s = [1] * len(self.shape)
        for k in range(len(s) - 2, -1, -1):
            s[k] = s[k + 1] * self.shape[k + 1]
        return tuple(s) if i is None else s[i]

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


class Library:
    """Counts the calls that get through; every one succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def world(qlin, monkeypatch):
    w = types.SimpleNamespace(device=0, lib=Library(), qlin=qlin)
    monkeypatch.setattr(qlin, "lib", lambda: w.lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: w.device, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    w.allocated_on = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: w.allocated_on.append(s) or contextlib.nullcontext())
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: Tensor(
        (shape,) if isinstance(shape, int) else tuple(shape), dtype, int(str(device).split(":")[1])))

    def cache(device, workspace=None):
        return qlin.KVCache(Tensor((4, 2, 2, 16 * 64), torch.uint8, device), Tensor((4, 2, 1, 2), torch.float32, device),
                            workspace=workspace)

    def batch(device):
        i32 = lambda *shape: Tensor(shape, torch.int32, device)  # noqa: E731
        return qlin.KVBatch(i32(2), i32(1), i32(1, 4), 1, 1, 10)

    w.cache, w.batch, w.rows = cache, batch, lambda device: Tensor((1, 2, 64), torch.bfloat16, device)
    return w


def test_calls_on_the_current_device(world):
    world.device = 1
    c, b, x = world.cache(1), world.batch(1), world.rows(1)
    c.append(b, x, x, q=x)
    c.attend(b, x)
    c.read(b)
    c.poll_status()
    assert world.lib.calls[-4:] == ["qlin_kv_append", "qlin_kv_attend", "qlin_kv_read", "qlin_kv_poll_status"]


def test_another_current_device_is_refused(world):
    """The library launches on the current device, and the handle of a default stream is that of the current
    device's: a cache elsewhere must not be followed from there."""
    world.device = 1
    c, b, x = world.cache(1), world.batch(1), world.rows(1)
    world.device, world.lib.calls[:] = 0, []
    for call in (lambda: world.cache(1), lambda: c.append(b, x, x, q=x), lambda: c.append(b, x, x, stream=7),
                 lambda: c.attend(b, x), lambda: c.attend(b, x, stream=7), lambda: c.read(b), lambda: c.poll_status(),
                 lambda: c.poll_status(stream=7)):
        with pytest.raises(ValueError, match="current device"):
            call()
    assert world.lib.calls == []


def test_a_stream_of_another_device_is_refused(world):
    c, b, x = world.cache(0), world.batch(0), world.rows(0)
    here, there = (types.SimpleNamespace(device_index=d, cuda_stream=7) for d in (0, 1))
    c.attend(b, x, stream=here)
    c.attend(b, x, stream=9)
    assert world.allocated_on == [7, 9]  # their outputs belong to the stream of the call
    world.lib.calls[:] = []
    for call in (lambda: c.append(b, x, x, stream=there), lambda: c.attend(b, x, stream=there), lambda: c.read(b, stream=there),
                 lambda: c.poll_status(stream=there)):
        with pytest.raises(ValueError, match="stream"):
            call()
    assert world.lib.calls == []


def test_a_shared_workspace_is_cleared_once(world):
    first = world.cache(0)
    assert world.lib.calls.count("qlin_kv_init_workspace") == 1
    second = world.cache(0, workspace=first.workspace)
    assert second.ws == first.ws and world.lib.calls.count("qlin_kv_init_workspace") == 1
    world.cache(0, workspace=Tensor((1 << 20,), torch.uint8, 0))  # fresh memory
    assert world.lib.calls.count("qlin_kv_init_workspace") == 2


def test_workspaces_that_do_not_fit_are_refused(world):
    def needs(c, n):  # what the library asks for
        n._obj.value = 4096
        return 0
    world.lib.qlin_kv_workspace_bytes = needs
    for memory in (Tensor((4000,), torch.uint8, 0), world.qlin.KVWorkspace(Tensor((4095,), torch.uint8, 0))):
        with pytest.raises(ValueError, match="too small"):
            world.cache(0, workspace=memory)
    with pytest.raises(ValueError, match="current device"):
        world.qlin.KVWorkspace(Tensor((5000,), torch.uint8, 1))
    world.device = 1
    there = world.qlin.KVWorkspace(Tensor((5000,), torch.uint8, 1))
    world.device = 0
    for memory in (Tensor((5000,), torch.uint8, 1), there):
        with pytest.raises(ValueError, match="one device"):
            world.cache(0, workspace=memory)
    world.cache(0, workspace=Tensor((4096,), torch.uint8, 0))
