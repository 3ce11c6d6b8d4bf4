"""Rows of logits on which a draw is easily wrong, against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import sample as SM

pytestmark = pytest.mark.gpu


def flat_tail(V, steps, bits):
    """A peak and V - 1 tokens of `steps` 2^-bits of it: logits, temperature and that weight."""
    T = np.float32(0.7)
    d = np.float32((bits - np.log2(steps)) * np.log(2.0) * np.float64(T))
    z = np.full(V, -d, np.float32)
    z[0] = 0.0
    return z, T, float(np.exp(-np.float64(d) / np.float64(T)))


@pytest.mark.parametrize("V,steps,bits", [(131073, 18, 45), (200001, 12, 45), (262145, 5, 44), (300000, 4, 44), (600000, 1, 43)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_flat_tail_far_below_the_peak_has_its_mass(V, steps, bits, dtype):
    """The tail's mass is about 1.1 to 1.4 times 2^-24 of the peak's, so u = 1 - 2^-24 falls into
    it, at token j with (V - 1) u - (1 - u) / w <= j.  A weight's error e moves that by
    e (1 - u) / w, at most e V: with e = 2^-30 (the kernel's) plus the distance of w from whole
    steps (2e-6 with these logits in fp32) less than a token."""
    from depth_planed_kv_b200.ripe import ripe_sample
    z, T, w = flat_tail(V, steps, bits)
    zd = torch.from_numpy(z).cuda()[None]
    u = np.float32(1 - 2.0 ** -24)
    if dtype == "bf16":   # the temperature carries what the logits cannot
        zd = zd.bfloat16()
        z = zd.float().cpu().numpy()[0]
        T = np.float32(-np.float64(z[1]) / ((bits - np.log2(steps)) * np.log(2.0)))
        w = float(np.exp(np.float64(z[1]) / np.float64(T)))
    assert abs(w * 2.0 ** bits / steps - 1) < 4e-6
    tok, lp = ripe_sample(zd, torch.tensor([u]).cuda(), torch.tensor([T]).cuda())
    ref, ref_lp, _ = SM.draw(z, float(u), float(T))
    assert ref > V // 20
    assert abs(int(tok) - ref) <= 1 + 4e-6 * V
    assert abs(float(lp) - ref_lp) <= 1e-5


@pytest.mark.parametrize("V", [131072, 131073, 262144, 262145, 1 << 20])
def test_equal_logits_at_the_edges_of_the_weights_width(V):
    """The sum of V largest weights is the largest there is."""
    from depth_planed_kv_b200.ripe import ripe_sample
    z = torch.zeros((3, V), device="cuda")
    u = torch.tensor([0.0, 0.5, 1 - 2.0 ** -24], device="cuda")
    one = torch.ones(3, device="cuda")
    for kw in ({}, dict(top_p=one * 0.99999), dict(min_p=one)):
        tok, lp = ripe_sample(z, u, **kw)
        kept = V if "top_p" not in kw else int(np.ceil(float(np.float32(0.99999)) * V))
        at = [int(np.floor(float(x) * kept)) for x in u.cpu().numpy().astype(np.float64)]
        assert list(tok.cpu().numpy()) == at and np.allclose(lp.cpu().numpy(), -np.log(kept), atol=1e-5)


@pytest.mark.parametrize("where", ["first eighth", "last eighth -inf", "middle", "falling", "rising"])
@pytest.mark.parametrize("V,n,dtype", [(3000, 12, "f32"), (32000, 6, "f32"), (65537, 4, "bf16"), (131072, 3, "f32")])
def test_large_logits_that_lie_together(V, n, dtype, where):
    """Whatever part of the vocabulary the large logits are in, with and without the filters; no
    margin of these seeds is below 1e-7, far above the weights' error."""
    from tests.test_sample_gpu import check
    rng = np.random.default_rng(V + len(where))
    z = (rng.standard_normal((n, V)) * 3).astype(np.float32)
    if where == "first eighth":
        z[:, :V // 8] += 12
    elif where == "last eighth -inf":
        z[:, V - V // 8:] = -np.inf
    elif where == "middle":
        z[:, V // 2:V // 2 + 150] += 25
    else:
        z = np.sort(z, 1) if where == "rising" else -np.sort(-z, 1)
    zd = torch.from_numpy(z).cuda()
    zd = zd.bfloat16() if dtype == "bf16" else zd
    one = np.ones(n, np.float32)
    u = rng.random(n).astype(np.float32)
    for k in (None, 3, 50, 200, 384, 1500):
        ks = None if k is None else np.full(n, k, np.int32)
        check(zd, u, one * np.float32(0.8), ks)
        check(zd, u, one * np.float32(0.8), ks, one * np.float32(0.9), one * np.float32(0.02))
