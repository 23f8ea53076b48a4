"""What a call allocates by itself belongs to the stream that it runs on: the
caching allocator orders a block's uses along one stream, so a block of
another stream can still be read or written by work that is pending there.
Without a GPU the library is a stand-in, and torch's allocations are noted with
the stream that is current when they are made."""
import contextlib

import pytest
import torch


class Side:
    """A stream by its handle, as torch.cuda.Stream has it."""
    cuda_stream = 0x5000


@pytest.fixture(scope="module")
def sp():
    from spatiotemporal_neural_field_b200 import build
    build.build()
    from spatiotemporal_neural_field_b200 import spin4d
    return spin4d


class FakeLib:
    """Every entry point succeeds; sizes are 64 bytes."""

    def __getattr__(self, name):
        return lambda *args: 64 if name.endswith(("_workspace", "_bytes")) else 0


@pytest.fixture
def seen(sp, monkeypatch):
    """[(kind, current stream)] of what is allocated, zeroed or read back."""
    log, current = [], [None]

    @contextlib.contextmanager
    def on(stream):
        before, current[0] = current[0], stream
        yield
        current[0] = before

    def note(owner, name):
        plain = getattr(owner, name)

        def noted(*args, **kw):
            log.append((name, current[0]))
            return plain(*args, **kw)
        monkeypatch.setattr(owner, name, noted)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "device", lambda index: contextlib.nullcontext())
    monkeypatch.setattr(sp, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(sp, "_current_device", lambda: -1)
    monkeypatch.setattr(sp, "lib", FakeLib())
    note(torch, "empty")
    note(torch, "zeros")
    note(torch.Tensor, "item")
    return log


def control(sp):
    c = object.__new__(sp.GradControl)
    c.device, c.index, c.address = torch.device("cpu"), -1, 1 << 20
    return c


def test_grad_norm_allocates_its_workspace_on_the_stream_of_the_call(sp, seen, monkeypatch):
    grads, ctl, side = sp.grad_list([]), control(sp), Side()
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    for stream, want in ((None, None), (side, side), (0x7000, ("external", 0x7000)), (0, "default"), (1, "default")):
        del seen[:]
        sp.grad_norm(grads, ctl, stream=stream)
        assert seen == [("empty", want)]
    del seen[:]
    sp.grad_norm(grads, ctl, workspace=torch.Tensor(8), stream=side)
    assert not seen                                     # the caller's is taken as it is


@pytest.mark.gpu
def test_a_freed_block_with_work_pending_is_not_the_workspace(sp):
    """A temporary of the workspace's size is freed while the sum over it still waits on the current stream; the norm on
    another stream leaves it alone, and both have their values."""
    g = torch.full((70_001,), 0.5, device="cuda")
    grads, ctl, side = sp.grad_list([g]), sp.grad_control(), torch.cuda.Stream()
    need = sp.grad_norm_workspace(1)
    sp.grad_norm(grads, ctl, max_norm=1.0, stream=side)      # the kernel is loaded before anything is pending
    for i in range(5):
        temporary = torch.full((need,), 3, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(4_000_000)                         # about 2 ms
        total = temporary.sum(dtype=torch.int64)
        del temporary
        sp.grad_norm(grads, ctl, max_norm=1.0, stream=side)
        torch.cuda.synchronize()
        assert int(total) == 3 * need
        assert int(ctl.step) == 2 + i and abs(float(ctl.norm) - (70_001 / 4) ** 0.5) <= 2.0 ** -24 * 200
