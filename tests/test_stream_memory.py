"""What a call allocates by itself belongs to the stream that it runs on: the
caching allocator orders a block's uses along one stream, so a block of
another stream can still be read or written by work that is pending there.
Without a GPU the library is a stand-in, and torch's allocations are noted with
the stream that is current when they are made."""
import contextlib

import pytest
import torch

from tests import tol


class Side:
    """Another library's stream object, known by its handle."""
    cuda_stream = 0x5000


SIDE = ("external", 0x5000)


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
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
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
    for stream, want in ((None, None), (side, SIDE), (0x7000, ("external", 0x7000)), (0, "default"), (1, "default")):
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


def calls(sp):
    """Every other call that allocates a workspace or outputs, by name: (call of a stream, allocations)."""
    t, i = torch.Tensor, lambda *shape: torch.Tensor(*shape).int()   # noqa: E731
    g, m = sp.GridDesc(L=2, F=2), sp.MlpDesc(in_dim=4, hidden=8, n_hidden=1)
    h, hx = sp.HeadsDesc(in_dim=4, hidden=8, sh_dim=48), sp.HexDesc()
    cam, desc = sp.camera([[1, 0, 0, 0], [0, 1, 0, 0], [0, 0, 1, 0]], 1, 1, 0, 0, 32, 16), sp.render_desc()
    pos, w = t(5, 4), t(9)
    hex_in = dict(mu=t(5, 3), frame=i(5), q_can=t(5, 4), logs_can=t(5, 3), sh_can=t(5, 48))
    scene = (t(5, 3), t(5, 6), t(5), t(5, 48))
    state = object.__new__(sp.RenderState)
    state.buf, state.max_pairs = torch.zeros(64, dtype=torch.uint8), 1 << 20
    return {
        "encode_fwd": (lambda s: sp.encode_fwd(g, pos, w, stream=s), 1),
        "decode_fwd": (lambda s: sp.decode_fwd(g, m, pos, w, w, stream=s), 5),
        "decode_bwd": (lambda s: sp.decode_bwd(g, m, pos, w, w, {}, w, w, stream=s), 1),
        "cov_assemble": (lambda s: sp.cov_assemble(t(5, 3), t(5, 4), stream=s), 1),
        "heads_fwd": (lambda s: sp.heads_fwd(g, h, pos, w, w, latent=True, raw=True, stream=s), 8),
        "heads_bwd": (lambda s: sp.heads_bwd(g, h, pos, w, w, {}, w, w, stream=s), 1),
        "hexplane_fwd": (lambda s: sp.hexplane_fwd(hx, hex_in, w, w, stream=s), 5),
        "hexplane_bwd": (lambda s: sp.hexplane_bwd(hx, hex_in, w, w, {}, w, w, stream=s), 1),
        "debug_corners": (lambda s: sp.debug_corners(g, pos, stream=s), 2),
        "morton_order": (lambda s: sp.morton_order(g, pos, stream=s), 3),
        "permute_rows": (lambda s: sp.permute_rows(w, i(5), stream=s), 1),
        "render_fwd": (lambda s: sp.render_fwd(cam, desc, *scene, stream=s), 2),
        "render_bwd": (lambda s: sp.render_bwd(cam, desc, *scene, t(3, 16, 32), state, stream=s), 4),
    }


@pytest.mark.parametrize("name", ["encode_fwd", "decode_fwd", "decode_bwd", "cov_assemble", "heads_fwd", "heads_bwd",
                                  "hexplane_fwd", "hexplane_bwd", "debug_corners", "morton_order", "permute_rows",
                                  "render_fwd", "render_bwd"])
def test_calls_allocate_on_the_stream_they_run_on(sp, seen, monkeypatch, name):
    call, count = calls(sp)[name]
    side = Side()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *device: Side())
    for stream, want in ((None, None), (side, SIDE)):
        del seen[:]
        call(stream)
        assert [w for _, w in seen] == [want] * count


@pytest.mark.gpu
def test_render_gradients_are_zeroed_on_the_stream_of_the_call(sp):
    """With work pending on the current stream the zeros still come before the kernel that adds to them."""
    cam, desc = sp.camera([[1, 0, 0, 0], [0, 1, 0, 0], [0, 0, 1, 3]], 40, 40, 30, 22, 60, 44), sp.render_desc()
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *shape: torch.rand(shape, device="cuda", generator=gen)   # noqa: E731
    cov = torch.tensor([1e-2, 0, 0, 1e-2, 0, 1e-2], device="cuda").repeat(200, 1)
    scene = (r(200, 3) - 0.5, cov, r(200) * 0.5 + 0.2, r(200, 48) - 0.5)
    image_grad, side = r(3, 44, 60), torch.cuda.Stream()
    _, state = sp.render(cam, desc, *scene)
    want = sp.render_bwd(cam, desc, *scene, image_grad, state)
    torch.cuda.synchronize()
    torch.cuda._sleep(4_000_000)
    got = sp.render_bwd(cam, desc, *scene, image_grad, state, stream=side)
    torch.cuda.synchronize()
    for k in want:
        # the same sums by atomics in another order: the bound that other tests have between two such runs
        assert bool(want[k].any())
        tol.normwise(got[k].cpu().numpy(), want[k].cpu().numpy(), 1e-4, k)


def test_render_reads_the_pair_count_on_the_stream_of_the_call(sp, seen, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *device: Side())
    cam, desc = sp.camera([[1, 0, 0, 0], [0, 1, 0, 0], [0, 0, 1, 0]], 1, 1, 0, 0, 32, 16), sp.render_desc()
    t, side = torch.Tensor, Side()
    for stream, want in ((None, None), (side, SIDE)):
        state = object.__new__(sp.RenderState)
        state.buf, state.max_pairs = torch.zeros(64, dtype=torch.uint8), 1 << 20
        del seen[:]
        sp.render(cam, desc, t(5, 3), t(5, 6), t(5), t(5, 48), state=state, stream=stream)
        assert [w for what, w in seen if what == "item"] == [want]


@pytest.mark.gpu
def test_render_on_a_stream_grows_its_state_and_gives_the_image(sp):
    """A state that is too small, on a stream with work pending: the pair count is read after the forward."""
    cam, desc = sp.camera([[1, 0, 0, 0], [0, 1, 0, 0], [0, 0, 1, 3]], 400, 400, 300, 220, 600, 440), sp.render_desc()
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *shape: torch.rand(shape, device="cuda", generator=gen)   # noqa: E731
    cov = torch.tensor([1e-1, 0, 0, 1e-1, 0, 1e-1], device="cuda").repeat(400, 1)
    scene = (r(400, 3) - 0.5, cov, r(400) * 0.5 + 0.2, r(400, 48) - 0.5)
    want, full = sp.render(cam, desc, *scene)
    few = (600 // 16 + 1) * (440 // 16 + 1)
    assert full.pairs_needed() > few
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    state = sp.RenderState(400, 600, 440, few, "cuda")
    state.buf.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(4_000_000)
    got, grown = sp.render(cam, desc, *scene, state=state, stream=side)
    torch.cuda.synchronize()
    assert grown is not state and grown.max_pairs == full.pairs_needed()
    assert torch.equal(got, want)


def test_probes_allocate_their_sinks_on_the_stream_they_run_on(sp, seen, monkeypatch):
    from spatiotemporal_neural_field_b200 import probe
    monkeypatch.setattr(probe, "lib", FakeLib())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *device: Side())
    buf, side = torch.Tensor(64), Side()
    for stream, want in ((None, None), (side, SIDE)):
        del seen[:]
        probe.probe_gather(buf, 4, 8, 1, stream=stream)
        probe.probe_stream(buf, 1, 1, stream=stream)
        probe.probe_fma(1, 1, "cpu", stream=stream)
        assert seen == [("zeros", want)] * 3


@pytest.mark.gpu
def test_streams_by_object_and_by_handle(sp):
    """A torch stream, another library's object with its handle, the handle itself, and the default stream's handles."""
    g = torch.full((5000,), 0.5, device="cuda")
    grads, ctl, side = sp.grad_list([g]), sp.grad_control(), torch.cuda.Stream()
    other = Side()
    other.cuda_stream = side.cuda_stream
    torch.cuda.synchronize()
    for i, stream in enumerate((side, other, side.cuda_stream, 0, 1)):
        sp.grad_norm(grads, ctl, max_norm=1.0, stream=stream)
        torch.cuda.synchronize()
        assert int(ctl.step) == 1 + i and abs(float(ctl.norm) - 1250 ** 0.5) <= 2.0 ** -24 * 64
