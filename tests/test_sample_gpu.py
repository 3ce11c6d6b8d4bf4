"""The token draw (ripe_sample) against the fp64 oracle.  Tokens have to be equal: the
kernel's weights are right to about 2^-32 of themselves and add up exactly, so a running
sum and its border would have to lie within about 1e-9 of each other to disagree; rows
closer than that are not drawn by these seeds (the test says so if one is).  logprob: a
few roundings to fp32 (2^-24 relative) of a value off by about 2^-32: 1e-6 relative and
1e-6 absolute cover it."""
import numpy as np
import pytest
import torch

from oracle import sample as SM

pytestmark = pytest.mark.gpu


def settings(rng, n, on):
    f = lambda x: x.astype(np.float32)
    t = f(np.where(rng.random(n) < 0.15, 0.0, 0.5 + rng.random(n))) if on[0] else None
    k = np.where(rng.random(n) < 0.3, 0, rng.integers(1, 300, n)).astype(np.int32) if on[1] else None
    p = f(np.where(rng.random(n) < 0.2, 1.0, 0.3 + 0.69 * rng.random(n))) if on[2] else None
    m = f(np.where(rng.random(n) < 0.3, 0.0, 0.2 * rng.random(n))) if on[3] else None
    return t, k, p, m


def check(z, u, t=None, k=None, p=None, m=None):
    from depth_planed_kv_b200.ripe import ripe_sample
    dev = lambda a: None if a is None else torch.as_tensor(np.ascontiguousarray(a)).cuda()
    zd = z if isinstance(z, torch.Tensor) else dev(z)
    tok, lp = ripe_sample(zd, dev(u), dev(t), dev(k), dev(p), dev(m))
    torch.cuda.synchronize()
    tok, lp = tok.cpu().numpy(), lp.cpu().numpy()
    zz = zd.float().cpu().numpy()
    for i in range(len(u)):
        pick = lambda a, off: off if a is None else a[i]
        ref, ref_lp, margin = SM.draw(zz[i], float(u[i]), float(pick(t, 1.0)), int(pick(k, 0)), float(pick(p, 1.0)),
                                      float(pick(m, 0.0)))
        assert tok[i] == ref, (i, tok[i], ref, margin)
        if np.isfinite(ref_lp):
            assert abs(lp[i] - ref_lp) <= 1e-6 + 1e-6 * abs(ref_lp), (i, lp[i], ref_lp)
        else:
            assert lp[i] == ref_lp
    return tok


ALL = [(0, 0, 0, 0), (1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1), (1, 1, 1, 1), (1, 1, 1, 0), (1, 0, 1, 1)]


@pytest.mark.parametrize("on", ALL, ids=str)
@pytest.mark.parametrize("V", [1, 2, 31, 333, 4097, 32000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_draw_matches_oracle(V, on, dtype):
    rng = np.random.default_rng(V + sum(b << i for i, b in enumerate(on)))
    n = 24
    z = torch.from_numpy((rng.standard_normal((n, V)) * rng.uniform(0.5, 6, (n, 1))).astype(np.float32)).cuda()
    if dtype == "bf16":
        z = z.bfloat16()
    check(z, rng.random(n).astype(np.float32), *settings(rng, n, on))


@pytest.mark.parametrize("V,n,dtype", [(131072, 6, "f32"), (65537, 9, "bf16"), (200001, 3, "f32"), (600000, 3, "bf16"),
                                       (450001, 2, "f32")])
def test_large_vocabularies(V, n, dtype):
    rng = np.random.default_rng(V)
    for on in ((1, 0, 0, 0), (1, 1, 1, 1), (0, 0, 1, 0)):
        z = torch.from_numpy((rng.standard_normal((n, V)) * 3).astype(np.float32)).cuda()
        if dtype == "bf16":
            z = z.bfloat16()
        check(z, rng.random(n).astype(np.float32), *settings(rng, n, on))


def test_rows_of_any_stride_and_alignment():
    rng = np.random.default_rng(3)
    z = torch.from_numpy(rng.standard_normal((7, 1201)).astype(np.float32)).cuda()
    for d in (torch.float32, torch.bfloat16):
        check(z.to(d)[:, 3:1000], rng.random(7).astype(np.float32), *settings(rng, 7, (1, 1, 1, 1)))


def test_ties_keep_the_lowest_index():
    n, V = 12, 5000
    rng = np.random.default_rng(4)
    z = np.zeros((n, V), np.float32)
    z[:, ::3] = 1.0       # two values only
    z[:, 7] = -0.0
    for k in (1, 2, 5, 1666, 1667, 1668, 4999):
        tok = check(z, rng.random(n).astype(np.float32), None, np.full(n, k, np.int32))
        assert (tok % 3 == 0).all() or k > 1667
    for p in (1e-6, 0.1, 0.4496, 0.5, 0.999):
        check(z, rng.random(n).astype(np.float32), None, None, np.full(n, p, np.float32))
        check(z, rng.random(n).astype(np.float32), None, np.full(n, 2000, np.int32), np.full(n, p, np.float32))
    # exact borders: equal weights, u and p on the steps
    z = np.full((4, 4), 2.0, np.float32)
    u = np.array([0.0, 0.25, 0.5, 0.75], np.float32)
    assert list(check(z, u)) == [0, 1, 2, 3]
    assert list(check(z, u, None, None, np.full(4, 0.5, np.float32))) == [0, 0, 1, 1]
    assert list(check(z, u, None, np.full(4, 3, np.int32), np.full(4, 0.5, np.float32))) == [0, 0, 1, 1]


def test_border_at_zero_and_at_minus_infinity():
    rng = np.random.default_rng(11)
    n, V = 6, 6000
    z = -np.abs(rng.standard_normal((n, V))).astype(np.float32) - 0.01
    z[:, 100:900] = 0.0
    z[:, 500] = -0.0
    z[:, :50] = 0.5
    u = rng.random(n).astype(np.float32)
    for k in (49, 50, 51, 849, 850, 851, 2000):
        check(z, u, None, np.full(n, k, np.int32))
        check(z, 1 - u / 100, None, np.full(n, k, np.int32), np.full(n, 0.99, np.float32))
    z[:, 2000:] = -np.inf
    for k in (1999, 2000, 2001, 5999):
        check(z, 1 - u / 1000, None, np.full(n, k, np.int32))
        check(z, 1 - u / 1000, None, np.full(n, k, np.int32), np.full(n, 0.999, np.float32))


def test_extreme_settings():
    rng = np.random.default_rng(5)
    n, V = 8, 3000
    z = (rng.standard_normal((n, V)) * 4).astype(np.float32)
    one = np.ones(n, np.float32)
    u = rng.random(n).astype(np.float32)
    for t in (1e-6, 1e-3, 30.0, 1e4):
        check(z, u, one * np.float32(t))
        check(z, u, one * np.float32(t), None, one * np.float32(0.9))
        check(z, u, one * np.float32(t), np.full(n, 2500, np.int32), one * np.float32(0.9))
    for m in (1.0, 2.0, 1e-30):
        check(z, u, None, None, None, one * np.float32(m))
    check(z, u, None, np.full(n, V + 5, np.int32), one * 0)
    check(z * 1000, u, None, None, one * np.float32(0.99))
    # u = 0: the first kept token of any weight, however small
    z[:, 0] = z.max(1) - 60
    tok = check(z, 0 * u)
    assert (tok == 0).all()
    check(z, 0 * u, None, None, one * np.float32(0.9))
    check(z, one - np.float32(2 ** -24))


def test_masked_logits():
    rng = np.random.default_rng(6)
    n, V = 10, 2500
    z = rng.standard_normal((n, V)).astype(np.float32)
    z[:, rng.random(V) < 0.9] = -np.inf
    z[0] = -np.inf               # nothing left
    z[1] = np.finfo(np.float32).min
    z[2] = np.nan
    z[3, :] = -np.inf
    z[3, 17] = -5.0              # one left
    z[4, 5] = np.nan
    u = rng.random(n).astype(np.float32)
    for on in ALL:
        tok = check(z, u, *settings(rng, n, on))
        assert tok[0] == -1 and tok[2] == -1 and tok[3] == 17
    z = rng.standard_normal((n, V)).astype(np.float32)
    z[:, 9] = z[:, 1200] = np.inf   # all the mass on two
    for on in ALL:
        tok = check(z, u, *settings(rng, n, on))
        assert set(tok) <= {9, 1200}


def test_frequencies_follow_the_kept_distribution():
    from depth_planed_kv_b200.ripe import ripe_sample
    rng = np.random.default_rng(7)
    z = rng.standard_normal(50).astype(np.float32) * 2
    n = 20000
    u = (np.arange(n, dtype=np.float64) / n).astype(np.float32)
    sel, w = SM.kept(z, 0.8, 20, 0.9, 0.01)
    tok, _ = ripe_sample(torch.from_numpy(np.tile(z, (n, 1))).cuda(), torch.from_numpy(u).cuda(),
                         torch.full((n,), 0.8).cuda(), torch.full((n,), 20, dtype=torch.int32).cuda(),
                         torch.full((n,), 0.9).cuda(), torch.full((n,), 0.01).cuda())
    got = np.bincount(tok.cpu().numpy(), minlength=50) / n
    ref = np.zeros(50)
    ref[sel] = w[sel] / w[sel].sum()
    # an even grid of u counts each share to within one grid step at either end
    assert np.abs(got - ref).max() <= 2.0 / n + 1e-6


def test_captured_and_on_another_stream():
    from depth_planed_kv_b200.ripe import ripe_sample
    rng = np.random.default_rng(8)
    z = torch.from_numpy(rng.standard_normal((16, 9000)).astype(np.float32)).cuda()
    u = torch.from_numpy(rng.random(16).astype(np.float32)).cuda()
    p = torch.full((16,), 0.8).cuda()
    ref = ripe_sample(z, u, top_p=p)[0].clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = ripe_sample(z, u, top_p=p, stream=s)[0]
    torch.cuda.synchronize()
    assert (got == ref).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ripe_sample(z, u, top_p=p)
    z.copy_(z.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    assert (out[0] == ripe_sample(z, u, top_p=p)[0]).all()
