"""The delta rule's, beam selection's and reordering's calls on other streams than torch's current one and in captured
graphs: what they make themselves is taken on the stream that they run on, and a replay gives what the calls give."""
import pytest
import torch

import selective_scan_gb300 as ss
from tests.gpu_util import device
from tests.util import assert_bits_equal

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
CU, LENGTHS, G, H, N, P = [0, 300, 300, 340], [300, 0, 40], 2, 4, 64, 40


def make(dev, seed=1):
    g = torch.Generator().manual_seed(seed)
    draw = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    rows = CU[-1]
    return dict(q=draw(rows, G, N).to(BF16).to(dev), k=draw(rows, G, N).to(BF16).to(dev), v=draw(rows, H, P).to(BF16).to(dev),
                g=(-draw(rows, H).abs() * 0.2).to(dev), beta=torch.sigmoid(draw(rows, H)).to(dev), state=draw(3, H, P, N).to(dev),
                dy=draw(rows, H, P).to(BF16).to(dev), logits=draw(6, 5000).to(dev), scores=-draw(2, 3).abs().to(dev),
                slots=torch.tensor([[1, 2, 0]], dtype=torch.int32, device=dev))


def empty(dev):
    e = lambda *s, t=BF16: torch.zeros(s, dtype=t, device=dev)  # noqa: E731
    rows = CU[-1]
    return dict(y=e(rows, H, P), kept=e(ss.gated_delta_rule_checkpoints(CU), H, P, N, t=F32), state=e(3, H, P, N, t=F32),
                dq=e(rows, G, N), dk=e(rows, G, N), dv=e(rows, H, P), dg=e(rows, H), dbeta=e(rows, H), ds=e(3, H, P, N, t=F32),
                scores=e(2, 3, t=F32), parents=e(2, 3, t=torch.int32), tokens=e(2, 3, t=torch.int32), status=e(1, t=torch.int32))


def chain(i, o, stream=None):
    """Everything once; the reordering by the first sequence's parents."""
    ss.gated_delta_rule(o["y"], i["q"], i["k"], i["v"], i["g"], i["beta"], o["state"], CU, [2, 0, 1], [1, 0, 0], l2_eps=1e-6,
                        checkpoints=o["kept"], stream=stream)
    ss.gated_delta_rule_backward(o["dq"], o["dk"], o["dv"], o["dg"], o["dbeta"], o["ds"], i["dy"], None, i["q"], i["k"], i["v"],
                                 i["g"], i["beta"], o["kept"], CU, l2_eps=1e-6, stream=stream)
    ss.beam_select(o["scores"], o["parents"], o["tokens"], i["logits"], i["scores"], stream=stream)
    ss.reorder_states([o["state"]], i["slots"], o["parents"][:1], o["status"], stream=stream)


def same(got, want):
    for k in want:
        assert_bits_equal(got[k].cpu(), want[k].cpu(), k)


def fresh_outputs(dev, i):
    o = empty(dev)
    o["state"].copy_(i["state"])
    return o


@pytest.mark.parametrize("form", ["stream", "handle", "default"])
def test_calls_beside_a_current_stream_that_is_still_busy(form):
    dev = device()
    i = make(dev)
    want, got = fresh_outputs(dev, i), fresh_outputs(dev, i)
    chain(i, want)
    torch.cuda.synchronize()
    sizes = [ss.gated_delta_rule_workspace_bytes(CU, H, P, N, G, BF16), ss.gated_delta_rule_workspace_bytes(CU, H, P, N, G, BF16, True),
             ss.library().mamba2_beam_select_workspace_bytes(2, 3, 3, 5000)]
    assert all(s > 0 for s in sizes)
    side = torch.cuda.Stream()
    stream = {"stream": side, "handle": side.cuda_stream, "default": 0}[form]
    busy = torch.cuda.Stream() if form == "default" else torch.cuda.current_stream()
    busy.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(busy):
        torch.cuda._sleep(50_000_000)
        written = [torch.zeros(s, dtype=torch.uint8, device=dev) for s in sizes]
        del written  # (their blocks are the ones that torch gives out next on this stream)
        chain(i, got, stream)
    torch.cuda.synchronize()
    same(got, want)


def test_a_captured_chain_replayed_on_other_values():
    """One graph, replayed with other inputs at the same addresses; another graph of the same calls between the replays."""
    dev = device()
    i, values = make(dev), [make(dev, 2), make(dev, 3)]
    outs = [fresh_outputs(dev, i), fresh_outputs(dev, i)]
    chain(i, outs[0])  # warm-up
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            chain(i, o)
        graphs.append(g)
    for v in values:
        for name in i:
            i[name].copy_(v[name])
        want = fresh_outputs(dev, i)
        chain(i, want)
        for o in outs:
            o["state"].copy_(i["state"])
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for o in outs:
            same(o, want)


def test_two_calls_at_once_on_two_streams():
    dev = device()
    ins = [make(dev, 4), make(dev, 5)]
    want = [fresh_outputs(dev, i) for i in ins]
    for i, o in zip(ins, want):
        chain(i, o)
    got = [fresh_outputs(dev, i) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for i, o, s in zip(ins, got, streams):
            with torch.cuda.stream(s):
                o["state"].copy_(i["state"])
                chain(i, o)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        same(a, b)


def test_no_wait_ran_out():
    device()
    assert ss.library().mamba2_device_timeouts() == 0
