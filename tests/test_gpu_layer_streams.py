"""Objects of the layer module made and called on a stream of their own while the current
one is busy: nothing that they do waits for it, and nothing of its comes late into them."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_route_amd import layer as LY
from nvfp4_block_scaled_route_amd import workloads as W

from .gpu_common import DEV, dev, host, say, upload_weights
from .test_gpu_expert_mlp import Step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True])
def test_routing_and_experts_on_a_stream_of_their_own(raw):
    """The current stream frees memory that its unfinished work still writes, and ends its
    work after the side stream's."""
    T, K, E, H, I, tile = 64, 4, 8, 136, 72, 32
    s = Step(T, K, E, H, I, tile, seed=21)
    s.forward()
    s.backward()
    want, meta = s.results(), s.routing.meta.clone()
    total = int(s.routing.total_rows.item())
    maps = [t.clone() for t in (s.routing.exp2perm, s.routing.perm2tok[:total], s.routing.expert_offsets, s.routing.expert_counts)]
    for t in (s.out, s.d_x, s.d_w13, s.d_w2, s.d_weights):
        t.fill_(float("nan"))
    sizes = [meta.numel() * 4, s.mlp.rows.nbytes, s.mlp.gate_up.nbytes, s.mlp.inter.nbytes]
    del meta
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    torch.cuda.synchronize()
    say("Routing and ExpertMlp on a side stream, raw", raw)
    junk = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(3)]
    torch.cuda._sleep(60_000_000)
    for t in junk:
        t.fill_(0xFF)
    done.record()
    del junk, t
    handle = side.cuda_stream if raw else side
    s.routing, s.mlp = LY.Routing(T, K, E, tile, stream=handle), LY.ExpertMlp(T, K, E, H, I, tile, stream=handle)
    s.forward(handle)
    s.backward(stream=handle)
    side.synchronize()
    say("the current stream has ended before it:", done.query())
    for a, b in zip(s.results(), want):         # (waits for both streams)
        assert torch.equal(a, b)
    r = s.routing
    for a, b in zip((r.exp2perm, r.perm2tok[:total], r.expert_offsets, r.expert_counts), maps):
        assert torch.equal(a, b)


@pytest.mark.parametrize("raw", [False, True])
def test_buffers_on_a_stream_of_their_own(raw):
    """The layer's, in the same way."""
    wl = W.WORKLOADS["tiny"]
    inp = W.make_inputs(wl)
    w = upload_weights(inp)
    x, gs, lg, nw = dev(inp.x_bf16), dev(inp.a1_gscale), dev(inp.logits), dev(inp.norm_weight_bf16)
    shape = LY.LayerShape(wl.T, wl.H, wl.I, wl.E, wl.K, wl.tile_m)

    def run(bufs, stream=None):
        LY.run_layer(bufs, x, gs, lg, None, None, w, nw, wl.gain_center, wl.eps, bool(wl.weight_before_norm), stream=stream)

    first = LY.Buffers(shape, DEV)
    run(first)
    torch.cuda.synchronize()
    want, size = {k: host(getattr(first, k)).copy() for k in ("ids", "weights", "meta", "out")}, first.workspace.nbytes
    first.check_sync()
    del first
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    torch.cuda.synchronize()
    say("Buffers on a side stream, raw", raw)
    junk = torch.empty(size, dtype=torch.uint8, device=DEV)
    torch.cuda._sleep(60_000_000)
    junk.fill_(0xFF)
    done.record()
    del junk
    handle = side.cuda_stream if raw else side
    bufs = LY.Buffers(shape, DEV, stream=handle)
    run(bufs, handle)
    side.synchronize()
    say("the current stream has ended before it:", done.query())
    torch.cuda.synchronize()
    bufs.check_sync()
    for k, v in want.items():
        assert np.array_equal(host(getattr(bufs, k)), v), k


@pytest.mark.parametrize("raw", [False, True])
def test_every_call_runs_on_the_stream_given(raw):
    """Two layers on two streams, with new inputs each time, everything that the calls write
    set to NaN or -1 before, and the current stream busy until they are done: a call that
    went there instead would come too late, and one that wrote nothing leave NaN."""
    steps = [Step(64, 4, 8, 136, 72, 32, seed=51), Step(300, 2, 4, 128, 264, 128, seed=52)]
    sides, done = [torch.cuda.Stream() for _ in steps], torch.cuda.Event()
    inputs = ("x", "d_out", "logits", "w13", "w2")

    def run(s, stream=None):
        s.forward(stream)
        s.backward(stream=stream)

    def written(s):
        m, r = s.mlp, s.routing
        return (s.out, s.d_x, s.d_w13, s.d_w2, s.d_weights, m.rows, m.gate_up, m.inter, m.out_rows, m.d_inter, m.d_rows, r.weights)

    before = [None, None]
    for it in range(3):
        want = []
        for i, s in enumerate(steps):
            g = torch.Generator(device=DEV)
            g.manual_seed(100 + 10 * it + i)
            for name in inputs:
                t = getattr(s, name)
                scale = t.shape[-1] ** -0.5 if name.startswith("w") else 1.0
                t.copy_(scale * torch.randn(t.shape, generator=g, device=DEV))
            run(s)
            want.append(s.results())
            if before[i] is not None:
                assert not any(torch.equal(a, b) for a, b in zip(want[i], before[i]))
            before[i] = want[i]
            for t in written(s):
                t.fill_(float("nan"))
            s.routing.meta.fill_(-1)
            s.routing.ids.fill_(-1)
        torch.cuda.synchronize()
        say("two layers on two streams, raw", raw, "time", it)
        torch.cuda._sleep(60_000_000)
        done.record()
        for s, side in zip(steps, sides):
            run(s, side.cuda_stream if raw else side)
        got = []
        for s, side in zip(steps, sides):
            with torch.cuda.stream(side):
                got.append([t.clone() for t in (s.out, s.d_x, s.d_w13, s.d_w2, s.d_weights)])
        for side in sides:
            side.synchronize()
        say("the current stream has ended before them:", done.query())
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for a, b in zip(g, w):
                assert torch.equal(a, b)
