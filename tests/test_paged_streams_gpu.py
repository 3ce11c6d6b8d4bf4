"""Calls of the serving operators on one stream beside calls on another, without a
synchronisation between them: each works in memory of its own stream."""
import numpy as np
import pytest
import torch

from tests.test_paged_gpu import Batch

pytestmark = pytest.mark.gpu


def test_a_call_on_the_current_stream_beside_one_on_another():
    from depth_planed_kv_b200.ripe import ripe_paged_attn
    # both leave partials in their work space, whose sizes are equal: a block of the first
    # call's, given back when it returns, would suit the second
    a, b = (Batch([9000, 700], new, 8, 2, 128, 16, seed=30 + i) for i, new in enumerate(([70, 200], [65, 40])))
    refs = [x.oracle() for x in (a, b)]
    devs = [x.dev() for x in (a, b)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a.out.fill_(77.0)
        for _ in range(3):
            ripe_paged_attn(a.q, a.k, a.v, *devs[0], a.out[:a.rows], a.lse[:a.rows], max_ntok=200)
            ripe_paged_attn(b.q, b.k, b.v, *devs[1], b.out[:b.rows], b.lse[:b.rows], max_ntok=65, stream=s)
        torch.cuda.synchronize()
        for x, (ref, ref_lse) in zip((a, b), refs):
            assert np.abs(x.out[:x.rows].float().cpu().numpy() - ref).max() < 0.05
            assert np.abs(x.lse[:x.rows].cpu().numpy() - ref_lse).max() < 2e-4
            assert bool((x.out[x.rows:] == 77.0).all())


def test_draws_on_two_streams():
    from depth_planed_kv_b200.ripe import ripe_accept, ripe_sample
    g = torch.Generator().manual_seed(31)
    z = torch.randn((40, 30000), generator=g).cuda() * 3
    u = torch.rand(40, generator=g).cuda()
    p = torch.full((40,), 0.9).cuda()
    want, want_lp = (t.clone() for t in ripe_sample(z, u, top_p=p))
    zp, zq = z.reshape(10, 4, -1), z.flip(0).reshape(10, 4, -1).contiguous()
    x1, ua = want.reshape(10, 4).contiguous(), torch.rand((10, 4, 3), generator=g).cuda()
    acc = [t.clone() for t in ripe_accept(zp, zq, None, x1, None, ua, 1.0)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = []
    for _ in range(30):
        # memory that the current stream has just given back, with a kernel of it still to run
        junk = torch.empty(40, dtype=torch.int32, device="cuda")
        torch.cuda._sleep(200000)
        junk.fill_(-5)
        del junk
        held.append((ripe_sample(z, u, top_p=p, stream=s), ripe_accept(zp, zq, None, x1, None, ua, 1.0, stream=s)))
    torch.cuda.synchronize()
    for (tok, lp), out in held:
        assert (tok == want).all() and (lp == want_lp).all()
        assert all((t == w).all() for t, w in zip(out, acc))


def test_a_side_stream_inside_a_captured_graph():
    """The work space and the outputs of calls on a stream that joined the capture belong to
    the graph."""
    from depth_planed_kv_b200.ripe import ripe_paged_attn, ripe_sample
    b = Batch([3000, 700], [70, 20], 8, 2, 128, 16, seed=33)
    z, u = torch.randn((20, 9000), device="cuda"), torch.rand(20, device="cuda")
    dev, s = b.dev(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        s.wait_stream(main)
        ripe_paged_attn(b.q, b.k, b.v, *dev, b.out[:b.rows], max_ntok=70, stream=s)
        tok, lp = ripe_sample(z, u, stream=s)
        main.wait_stream(s)
    ref, _ = b.oracle()
    for _ in range(3):
        b.out.fill_(77.0)
        z.copy_(torch.randn(z.shape))
        graph.replay()
        eager, _ = ripe_sample(z, u)
        other = torch.randn((1 << 20,), device="cuda")   # what is free is used by others meanwhile
        torch.cuda.synchronize()
        assert np.abs(b.out[:b.rows].float().cpu().numpy() - ref).max() < 0.05 and (tok == eager).all()
        del other
