"""The recurrent block's operators on a stream that is not torch's current one: where their workspaces come from (on
the CPU, with a stand-in for torch's streams), and their results while freed memory of the current stream is still in
use there."""
import contextlib

import pytest
import torch

import selective_scan_gb300 as ss
from tests.gpu_util import device
from tests.util import assert_bits_equal


class _Handle:
    """A stream of another library: all that it shows is its handle."""
    cuda_stream = 0x5000


class _Stop(Exception):
    pass


@pytest.fixture
def streams(monkeypatch):
    """torch.cuda's streams replaced by names; a list of the ones that were current when memory was taken."""
    now, taken = ["the caller's"], []

    @contextlib.contextmanager
    def stream(s):
        before, now[0] = now[0], s
        try:
            yield
        finally:
            now[0] = before

    class Memory:
        def record_stream(self, s):
            pass

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return 0x100

        def numel(self):
            return 64

        def element_size(self):
            return 1

    def empty(*_, **__):
        taken.append(now[0])
        return Memory()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch, "empty", empty)
    return now, taken


@pytest.mark.parametrize("stream,where", [(None, "the caller's"), (0x7000, ("external", 0x7000)), (0, "default"),
                                          (_Handle(), ("external", 0x5000))], ids=["none", "handle", "zero", "object"])
def test_a_workspace_is_taken_on_the_stream_that_uses_it(streams, stream, where):
    """Memory that the current stream has freed may still be in use there, so only that stream's order allows its
    reuse. (0 is the legacy default stream's handle.)"""
    now, taken = streams
    assert ss._workspace(64, None, "cuda", stream)[:2] == (0x100, 64)
    assert taken == [where] and now == ["the caller's"]


@pytest.mark.parametrize("stream,where", [(None, "the caller's"), (0x7000, ("external", 0x7000)), (0, "default")],
                         ids=["none", "handle", "zero"])
def test_the_block_runs_on_the_stream_that_it_is_given(streams, monkeypatch, stream, where):
    """Its operators run on torch's current stream, so that has to be the stream asked for, also for handle 0."""
    from selective_scan_gb300 import recurrent_block
    now, _ = streams
    ran = []

    def add_rmsnorm(*_, **__):
        ran.append(now[0])
        raise _Stop

    monkeypatch.setattr(recurrent_block, "add_rmsnorm", add_rmsnorm)
    w = torch.zeros((8, 16), dtype=torch.bfloat16)
    block = recurrent_block.RecurrentBlock(recurrent_block.RecurrentBlockWeights(
        norm_w=None, w_x=w, b_x=None, w_gate=w, b_gate=None, lower=None, w_out=None, b_out=None))
    with pytest.raises(_Stop):
        block.prefill(w, None, None, [0, 8], [0], [1], stream=stream)
    assert ran == [where] and now == ["the caller's"]


def test_the_scans_workspaces_are_taken_there_too(streams, monkeypatch, product_lib):
    import workloads as W
    asked = []

    def workspace(need, given, device, stream):
        asked.append((need > 0, given, stream))
        raise _Stop

    monkeypatch.setattr(ss, "_workspace", workspace)
    d = W.DIMS_130M
    z, x = torch.zeros((4096, d.d_inner), dtype=torch.bfloat16), torch.zeros((4096, d.conv_dim), dtype=torch.bfloat16)
    state, batch = torch.zeros(1), ([0, 4096], [0], [1])
    with pytest.raises(_Stop):
        ss.ssd_scan(z, x, z, None, None, None, state, d, *batch, stream=0x7000)
    with pytest.raises(_Stop):
        ss.prefill_host(z, x, z, z, None, None, None, None, None, None, 1, 1e-5, state, state, d, *batch, stream=0x7000)
    assert asked == [(True, None, 0x7000)] * 2


@pytest.mark.parametrize("stream,where", [(None, "the caller's"), (0x7000, ("external", 0x7000)), (0, "default")],
                         ids=["none", "handle", "zero"])
def test_the_layer_and_the_padded_batch_run_on_the_stream_that_they_are_given(streams, monkeypatch, product_lib, stream,
                                                                              where):
    """Their intermediates, and torch's copies of strided inputs, belong to the stream of the kernels that use them."""
    import workloads as W
    from selective_scan_gb300 import layer, padded
    now, _ = streams
    d, ran = W.DIMS_TINY, []

    def kernel(*_, **__):
        ran.append(now[0])
        raise _Stop

    for module, name in ((layer, "in_proj"), (padded, "pack_rows"), (padded, "decode_step")):
        monkeypatch.setattr(module, name, kernel)
    w = padded.Mamba2Weights(*[None] * 6)
    one = layer.Mamba2Layer(torch.zeros((1, 8)), None, w, d)
    x, z, dt = torch.zeros((2, 3, d.conv_dim)), torch.zeros((2, 3, d.d_inner)), torch.zeros((2, 3, d.heads))
    for call in (lambda: one.prefill(x[0], None, None, [0, 3], [0], [1], stream=stream),
                 lambda: one.decode(x[0], None, None, [0, 1, 2], stream=stream),
                 lambda: padded.forward(x, z, dt, w, d, padded.Mamba2Cache(None, None, [0, 1]), stream=stream),
                 lambda: padded.decode(x[:, 0], z[:, 0], dt[:, 0], w, d, padded.Mamba2Cache(None, None, [0, 1]), stream=stream)):
        with pytest.raises(_Stop):
            call()
    assert ran == [where] * 4 and now == ["the caller's"]


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["stream", "handle", "default"])
def test_operators_beside_a_current_stream_that_is_still_busy(form):
    """Every operator that takes a workspace of its own, on a stream that is not current, while the current stream
    still has to write memory that was freed on it: the results are those of the current stream alone."""
    dev = device()
    g = torch.Generator().manual_seed(1)
    draw = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    lengths, dim, n = [700, 0, 300], 136, 256
    cu = [0, 700, 700, 1000]
    x, gate, dy = (draw(1000, dim).bfloat16().to(dev) for _ in range(3))
    lower, pool, nw = torch.rand(dim, generator=g).to(dev), draw(3, dim).to(dev), draw(dim).to(dev)
    w, dyl, pre = draw(n, dim).bfloat16().to(dev), draw(1000, n).bfloat16().to(dev), draw(1000, n).bfloat16().to(dev)
    kept_rows = ss.gated_recurrence_checkpoints(cu)

    def outputs():
        e = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device=dev)  # noqa: E731
        f = torch.float32
        return dict(st=pool.clone(), y=e(1000, dim), kept=e(kept_rows, dim, t=f), dx=e(1000, dim), dg=e(1000, dim),
                    dlo=e(dim, t=f), ds=e(1000, dim), dnw=e(dim, t=f), dn=e(1000, dim), dw=e(n, dim), db=e(n, t=f))

    def chain(o, stream):
        ss.gated_recurrence(o["y"], x, gate, lower, o["st"], cu, [2, 0, 1], [1, 1, 0], checkpoints=o["kept"], stream=stream)
        ss.gated_recurrence_backward(o["dx"], o["dg"], o["dlo"], None, dy, None, x, gate, lower, o["kept"], cu, stream=stream)
        ss.add_rmsnorm_backward(o["ds"], None, o["dnw"], dy, None, x, nw, 1e-5, stream=stream)
        ss.linear_backward(o["dn"], o["dw"], o["db"], dyl, x, w, activation="silu", pre=pre, stream=stream)

    want, got = outputs(), outputs()
    chain(want, None)
    torch.cuda.synchronize()
    sizes = [ss.gated_recurrence_workspace_bytes(cu, dim), ss.gated_recurrence_workspace_bytes(cu, dim, True),
             ss.library().mamba2_add_rmsnorm_backward_workspace_bytes(1000, dim),
             ss.library().mamba2_linear_backward_workspace_bytes(1000, dim, n)]
    side = torch.cuda.Stream()
    stream = {"stream": side, "handle": side.cuda_stream, "default": 0}[form]
    busy = torch.cuda.Stream() if form == "default" else torch.cuda.current_stream()
    busy.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(busy):
        torch.cuda._sleep(50_000_000)
        written = [torch.zeros(s, dtype=torch.uint8, device=dev) for s in sizes]
        del written  # (their blocks are the ones that torch gives out next on this stream)
        chain(got, stream)
    torch.cuda.synchronize()
    for k in want:
        assert_bits_equal(got[k], want[k], k)
