"""A decoding loop over the paged cache as a server runs it, against the fp64 oracles: two
prompts written and attended to in chunks, single-token steps, then draft blocks whose
tokens ripe_sample draws, ripe_accept checks and the cache keeps or drops (a dropped
token's slot is simply written again).  Rejected tokens must leave no trace."""
import numpy as np
import pytest
import torch

from oracle import accept as AC
from oracle import paged as PG
from oracle import sample as SM

pytestmark = pytest.mark.gpu

H, HKV, D, PAGE, VOCAB = 8, 2, 64, 16, 300
TOL = 2 ** -8 * 2 + 2 ** -12  # of the largest value: one rounding of the weights, one of the output


def _i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


class Loop:
    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)
        n = 40
        self.k = torch.full((n, HKV, PAGE, D), float("nan"), dtype=torch.bfloat16, device="cuda")  # never-written slots
        self.v = self.k.clone()
        self.table = torch.randperm(n, generator=self.g).to(torch.int32)[:2 * 16].reshape(2, 16)
        self.ctx = [0, 0]
        self.vmax = 0.0

    def rand(self, n, heads):
        return torch.randn((n, heads, D), generator=self.g).to(torch.bfloat16)

    def step(self, new):
        """Appends and attends to `new` random tokens per sequence; returns O and checks it."""
        from depth_planed_kv_b200.ripe import ripe_paged_append, ripe_paged_attn
        rows = sum(new)
        row0 = np.concatenate([[0], np.cumsum(new)])
        K, V, Q = self.rand(rows, HKV), self.rand(rows, HKV), self.rand(rows, H)
        self.vmax = max(self.vmax, float(V.float().abs().max()))
        table, ctx, r0 = self.table.cuda(), _i32(self.ctx), _i32(row0)
        O = torch.empty((rows, H, D), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((rows, H), device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        ripe_paged_append(K.cuda(), V.cuda(), self.k, self.v, table, ctx, r0, err=err)
        ripe_paged_attn(Q.cuda(), self.k, self.v, table, ctx, r0, O, lse, max_ntok=max(new), err=err)
        torch.cuda.synchronize()
        assert int(err) == 0
        ref, ref_lse = PG.attn(Q.float().numpy(), self.k.float().cpu().numpy(), self.v.float().cpu().numpy(),
                               self.table.numpy(), self.ctx, row0)
        assert np.isfinite(ref).all()
        assert np.abs(O.float().cpu().numpy() - ref).max() <= TOL * self.vmax
        assert np.abs(lse.cpu().numpy() - ref_lse).max() <= 2e-4
        return O


@pytest.mark.parametrize("temperature", [0.0, 0.9])
def test_prompt_steps_drafts(temperature):
    from depth_planed_kv_b200.ripe import ripe_accept, ripe_sample
    loop = Loop(int(temperature * 10))
    head = torch.randn((H * D, VOCAB), generator=loop.g).cuda() * 0.3
    logits = lambda o, scale=1.0: (o.float().reshape(-1, H * D) @ head) * scale  # noqa: E731
    # prompts of 70 and 33 tokens in chunks of 32
    for new in ([32, 32], [32, 1], [6, 0]):
        loop.step(new)
        loop.ctx = [c + n for c, n in zip(loop.ctx, new)]
    assert loop.ctx == [70, 33]
    rng = np.random.default_rng(3)
    settings = dict(temperature=torch.full((2,), temperature).cuda(), top_k=_i32([20, 50]),
                    top_p=torch.full((2,), 0.95).cuda(), min_p=torch.full((2,), 0.02).cuda())
    # single tokens
    for _ in range(3):
        z = logits(loop.step([1, 1]))
        u = rng.random(2).astype(np.float32)
        tok, _ = ripe_sample(z, torch.from_numpy(u).cuda(), **settings)
        for i in range(2):
            ref, _, _ = SM.draw(z[i].cpu().numpy(), float(u[i]), temperature, (20, 50)[i], float(np.float32(0.95)), float(np.float32(0.02)))
            assert int(tok[i]) == ref
        loop.ctx = [c + 1 for c in loop.ctx]
    # draft blocks of 4: drawn from the draft's logits, checked against the final ones
    k, seen = 4, set()
    for _ in range(6):
        o = loop.step([k, k])
        zp = logits(o).reshape(2, k, VOCAB)
        zq = zp + torch.randn(zp.shape, generator=loop.g).cuda() * 0.7
        u = torch.from_numpy(rng.random(2 * k).astype(np.float32)).cuda()
        x1, _ = ripe_sample(zq.reshape(2 * k, VOCAB), u, temperature=torch.full((2 * k,), temperature).cuda())
        ua = rng.random((2, k, 3)).astype(np.float32)
        n_acc, tok, _ = ripe_accept(zp.contiguous(), zq.contiguous(), None, x1.reshape(2, k), None, torch.from_numpy(ua).cuda(),
                                    temperature)
        for b in range(2):
            if temperature == 0:   # greedy: no border to be near
                want = AC.accept_block(zp[b].cpu().numpy().astype(np.float64), zq[b].cpu().numpy().astype(np.float64), None,
                                       x1.reshape(2, k)[b].cpu().numpy(), np.zeros(k, int), ua[b].astype(np.float64), 0.0)
                assert (int(n_acc[b]), int(tok[b])) == want[:2]
        seen.update(n_acc.tolist())
        loop.ctx = [c + int(n) for c, n in zip(loop.ctx, n_acc)]  # the rejected tokens' slots are written again
    assert len(seen) > 1


def test_loop_step_in_one_graph():
    """append, attention and draw of a decode step captured once and replayed as the
    sequences grow; only the device-side lengths change."""
    from depth_planed_kv_b200.ripe import ripe_paged_append, ripe_paged_attn, ripe_sample
    loop = Loop(7)
    loop.step([20, 45])
    loop.ctx = [20, 45]
    head = torch.randn((H * D, VOCAB), generator=loop.g).cuda()
    table, ctx, r0 = loop.table.cuda(), _i32(loop.ctx), _i32([0, 1, 2])
    K, V, Q = (torch.zeros((2, n, D), dtype=torch.bfloat16, device="cuda") for n in (HKV, HKV, H))
    O = torch.empty((2, H, D), dtype=torch.bfloat16, device="cuda")
    u = torch.zeros(2, device="cuda")
    p = torch.full((2,), 0.9).cuda()

    def step():
        ripe_paged_append(K, V, loop.k, loop.v, table, ctx, r0)
        ripe_paged_attn(Q, loop.k, loop.v, table, ctx, r0, O, max_ntok=1)
        return ripe_sample(O.float().reshape(2, H * D) @ head, u, top_p=p)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tok, _ = step()
    for i in range(20):
        for t, n in ((K, HKV), (V, HKV), (Q, H)):
            t.copy_(loop.rand(2, n))
        u.copy_(torch.rand(2, generator=loop.g))
        ctx.copy_(torch.tensor(loop.ctx, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        ref, _ = PG.attn(Q.float().cpu().numpy(), loop.k.float().cpu().numpy(), loop.v.float().cpu().numpy(), loop.table.numpy(),
                         loop.ctx, [0, 1, 2])
        assert np.abs(O.float().cpu().numpy() - ref).max() <= TOL * 5
        z = (O.float().reshape(2, H * D) @ head).cpu().numpy()
        for b in range(2):
            want, _, margin = SM.draw(z[b], float(u[b]), 1.0, 0, float(np.float32(0.9)))
            assert int(tok[b]) == want, margin
        loop.ctx = [c + 1 for c in loop.ctx]
