"""CPU tests of what the prepared calls hold on to, and of the streams that the
8-bit calls run on: a library and tensors that stand in for the real ones, so
that no GPU is touched."""
import pytest

import linear_wl_forward_b200 as wl


class FakeTensor:
    """Enough of a CUDA tensor for the argument checks."""
    is_cuda = True
    device = None

    def __init__(self, *shape):
        self.shape = shape
        self.streams = []

    def data_ptr(self):
        return 1 << 20

    def record_stream(self, stream):
        self.streams.append(stream)


class FakeLib:
    def __init__(self):
        self.launched = []

    def wl_stacked_forward_fp8_workspace(self, *args):
        return 0

    def wl_plan_stacked_forward_fp8(self, *args):
        return 0

    def wl_run_fp8_plan(self, plan, stream):
        self.launched.append(stream)
        return 0

    def wl_stacked_forward_prefetch(self, *args):
        self.launched.append(args[-1])
        return 0

    def wl_free_fp8_plan(self, plan):
        pass


class NoDevice:
    index = 0


class Nothing:
    def __init__(self, *args):
        pass

    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


@pytest.fixture
def fake(monkeypatch):
    import torch

    fake = FakeLib()
    monkeypatch.setattr(wl, "lib", lambda: fake)
    monkeypatch.setattr(wl, "_lib", fake)
    monkeypatch.setattr(wl, "_need_cuda", lambda t, name: NoDevice)
    monkeypatch.setattr(wl, "_On", Nothing)
    monkeypatch.setattr(wl, "_ptr_on", lambda device, t, *rest: t.data_ptr())
    monkeypatch.setattr(wl, "_dev_ptr", lambda t, *rest: t.data_ptr())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: handle)
    return fake


def call():
    x = FakeTensor(3, 64)
    proj = [FakeTensor(40, 64), FakeTensor(1, 4), FakeTensor(40), FakeTensor(40, 8), FakeTensor(64, 8)]
    return x, proj, FakeTensor(3, 40)


def held(handle):
    """Every tensor that the handle's attributes lead to through tuples."""
    found, todo = [], list(vars(handle).values())
    while todo:
        v = todo.pop()
        if isinstance(v, FakeTensor):
            found.append(v)
        elif isinstance(v, tuple):
            todo.extend(v)
    return found


def test_fp8_handle_keeps_the_tensors_and_not_the_lists(fake):
    x, proj, y = call()
    tensors, projs, ys = [x, *proj, y], [proj], [y]
    handle = wl.prepare_stacked_fp8(x, projs, ys=ys)
    projs.clear()
    proj.clear()
    ys.clear()
    assert all(any(t is h for h in held(handle)) for t in tensors)
    out = handle(stream=5)
    assert out == [y] and fake.launched == [5]
    out[0] = None
    assert handle(stream=5) == [y] and handle.ys == [y]


def test_fp8_handle_records_each_stream_once(fake, monkeypatch):
    x, proj, y = call()
    ws = FakeTensor(100)
    monkeypatch.setattr(wl, "_workspace", lambda nbytes, device: ws)
    handle = wl.prepare_stacked_fp8(x, [proj], ys=[y])
    for stream in (5, 5, 9, 5, 9):
        handle(stream=stream)
    assert fake.launched == [5, 5, 9, 5, 9]
    assert all(t.streams == [5, 9] for t in (x, *proj, y, ws))


def test_bf16_handle_keeps_the_tensors_and_not_the_lists(fake, monkeypatch):
    monkeypatch.setattr(wl, "prefetch_ranges", lambda items: (None, 0))
    x, proj, y = call()
    proj, ahead = [FakeTensor(40, 64), *proj[2:]], FakeTensor(16)
    tensors, projs, ys, prefetch = [x, *proj, y, ahead], [proj], [y], [ahead]
    handle = wl.prepare_stacked(x, projs, ys=ys, prefetch=prefetch)
    for a in (projs, proj, ys, prefetch):
        a.clear()
    assert all(any(t is h for h in held(handle)) for t in tensors)
    out = handle(stream=5)
    assert out == [y] and fake.launched == [5]
    out[0] = None
    assert handle(stream=5) == [y] and handle.ys == [y]


def test_raw_handle_0_is_the_default_stream(monkeypatch):
    import torch

    device = torch.device("cuda", 3)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: ("external", handle, device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: ("default", device))
    entered = []

    class Enter(Nothing):
        def __init__(self, what):
            entered.append(what)

    monkeypatch.setattr(torch.cuda, "device", Enter)
    monkeypatch.setattr(torch.cuda, "stream", Enter)
    for handle, want in ((0, ("default", device)), (5, ("external", 5, device))):
        with wl._On(device, handle):
            assert entered[-1] == want
