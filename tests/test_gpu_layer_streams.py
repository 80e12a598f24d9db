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
