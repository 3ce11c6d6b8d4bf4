"""Batches that a paged call has to sort out on the device: sequences that are skipped,
and what that leaves of the others.  Tolerances as in test_paged_gpu.py (0.05 is several
times them for these values, and far below what a wrong key does)."""
import numpy as np
import pytest
import torch

from oracle import paged as PG
from tests.test_paged_gpu import Batch

pytestmark = pytest.mark.gpu


def bad_batch(b, what):
    """The batch's device arrays with sequence 1 spoilt; the code the calls report, and the
    sequences that they still serve."""
    table, ctx, row0 = b.dev()
    last = (b.ctx[1] + b.new[1] - 1) // b.page
    if what == "ctx":
        ctx[1] = table.shape[1] * b.page - b.new[1] + 1
    elif what == "neg":
        ctx[1] = -1
    elif what == "descend":   # sequence 2 would then claim a row of sequence 0
        row0[2] = row0[1] - 1
    elif what == "past":
        row0[2:] = b.rows + 1
    elif what == "negrow":
        row0[0] = -1
    elif what == "page":
        table[1, last] = b.k.shape[0]
    elif what == "negpage":
        table[1, last] = -1
    code = {"ctx": 2, "neg": 2, "descend": 8, "past": 8, "negrow": 8, "page": 9, "negpage": 9}[what]
    good = {"ctx": [0, 2], "neg": [0, 2], "descend": [0], "past": [0], "negrow": [1, 2], "page": [0, 2], "negpage": [0, 2]}[what]
    return (table, ctx, row0), code, good


WHAT = ["ctx", "neg", "descend", "past", "negrow", "page", "negpage"]


@pytest.mark.parametrize("what", WHAT)
@pytest.mark.parametrize("new", [[2, 3, 1], [20, 60, 30]], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_of_bad_sequences(dtype, new, what):
    """The pages hold the served sequences' new tokens and are otherwise as before."""
    from depth_planed_kv_b200.ripe import ripe_paged_append
    b = Batch([20, 30, 40], new, 4, 2, 64, 16, dtype, seed=40)
    dev, code, good = bad_batch(b, what)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = (torch.randn((b.rows, 2, 64)).to(b.dtype).cuda() for _ in range(2))
    rk, rv = b.k.cpu().float().numpy().copy(), b.v.cpu().float().numpy().copy()
    kn, vn = k.float().cpu().numpy(), v.float().cpu().numpy()
    for i in range(3):
        for j in range(b.new[i]):
            pos, r = b.ctx[i] + j, b.row0[i] + j
            if i in good or (code == 9 and pos // b.page != (b.ctx[1] + b.new[1] - 1) // b.page):
                rk[int(b.table[i, pos // b.page]), :, pos % b.page] = kn[r]
                rv[int(b.table[i, pos // b.page]), :, pos % b.page] = vn[r]
    ripe_paged_append(k, v, b.k, b.v, *dev, err=err)
    torch.cuda.synchronize()
    assert int(err) == code
    assert (b.k.float().cpu().numpy() == rk).all() and (b.v.float().cpu().numpy() == rv).all()


@pytest.mark.parametrize("what", WHAT)
@pytest.mark.parametrize("new,dtype", [([2, 3, 1], "bf16"), ([20, 60, 30], "bf16"), ([400, 300, 700], "bf16"),
                                       ([2, 3, 1], "f32"), ([40, 60, 30], "f32")], ids=str)
def test_attention_of_bad_sequences(new, dtype, what):
    """The served sequences' rows are right; the skipped ones' are left as they were (a bad
    page is read as page 0, so those rows mean nothing)."""
    from depth_planed_kv_b200.ripe import ripe_paged_attn
    b = Batch([20, 30, 40], new, 4, 2, 64, 16, dtype, seed=41)
    ref, ref_lse = b.oracle()
    dev, code, good = bad_batch(b, what)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ripe_paged_attn(b.q, b.k, b.v, *dev, b.out[:b.rows], b.lse[:b.rows], max_ntok=max(new), err=err)
    torch.cuda.synchronize()
    assert int(err) == code
    o, lse = b.out.float().cpu().numpy(), b.lse.cpu().numpy()
    for i in range(3):
        r = slice(int(b.row0[i]), int(b.row0[i + 1]))
        if i in good:
            assert np.abs(o[r] - ref[r]).max() < 0.05 and np.abs(lse[r] - ref_lse[r]).max() < 2e-4
        elif code != 9:
            assert (o[r] == 77.0).all() and (lse[r] == 77.0).all()
    assert (o[b.rows:] == 77.0).all()


@pytest.mark.parametrize("nseq,at", [(3, 1), (200, 0), (200, 137), (1024, 600), (1024, 1023)])
@pytest.mark.parametrize("most", [1, 40])
def test_offsets_that_descend_among_many_sequences(nseq, at, most):
    """All before the first such sequence is served, nothing from it on."""
    from depth_planed_kv_b200.ripe import ripe_paged_append, ripe_paged_attn
    rng = np.random.default_rng(nseq + at)
    new = rng.integers(1, most + 1, nseq)
    b = Batch(rng.integers(0, 40, nseq), new, 2, 1, 64, 16, seed=42)
    table, ctx, row0 = b.dev()
    row0[at + 1] = row0[at] - 1
    if at + 4 < nseq:
        row0[at + 3] = 0   # a second time, and rows of the first ones claimed once more
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kn = torch.randn((b.rows, 1, 64)).to(b.dtype).cuda()
    rk, kf = b.k.float().cpu().numpy().copy(), kn.float().cpu().numpy()
    for i in range(at):
        for j in range(new[i]):
            pos = b.ctx[i] + j
            rk[int(b.table[i, pos // 16]), :, pos % 16] = kf[b.row0[i] + j]
    ripe_paged_append(kn, kn, b.k, b.v, table, ctx, row0, err=err)
    torch.cuda.synchronize()
    assert int(err) == 8 and (b.k.float().cpu().numpy() == rk).all()
    err.zero_()
    ripe_paged_attn(b.q, b.k, b.v, table, ctx, row0, b.out[:b.rows], b.lse[:b.rows], max_ntok=most, err=err)
    torch.cuda.synchronize()
    assert int(err) == 8
    ref, _ = b.oracle()
    end = int(b.row0[at])
    o = b.out.float().cpu().numpy()
    assert end == 0 or np.abs(o[:end] - ref[:end]).max() < 0.05
    assert (o[end:] == 77.0).all()


RELEASED = [  # ctx, new, H, Hkv, d, dtype
    ([700, 45, 1300], [1, 1, 1], 4, 2, 64, "bf16"),
    ([700, 45, 1300], [3, 8, 2], 4, 2, 128, "bf16"),
    ([700, 45, 1300], [40, 9, 200], 4, 2, 96, "bf16"),
    ([700, 300, 1300], [400, 130, 20], 2, 2, 64, "bf16"),
    ([2000], [33], 16, 1, 32, "bf16"),
    ([700, 45, 1300], [1, 30, 2], 4, 2, 80, "bf16"),
    ([700, 45, 600], [2, 1, 40], 4, 2, 64, "f32"),
]


@pytest.mark.parametrize("case", RELEASED, ids=str)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 0), (70, 5), (33, 64), (250, 37)])
def test_pages_behind_the_window_may_be_given_back(case, page, window, sinks):
    """The table has no page any more where no token looks, and the pages that were there (and
    page 0) hold NaN."""
    from depth_planed_kv_b200.ripe import ripe_paged_attn
    b = Batch(*case[:5], page, case[5], seed=43)
    ref, ref_lse = b.oracle(window=window, sinks=sinks)
    table, ctx, row0 = b.dev()
    gone = []
    for i, c in enumerate(b.ctx):
        for p in range(table.shape[1]):
            # all its positions behind the first new token's window, none among the first
            if (p + 1) * page <= c + 1 - window and p * page >= sinks:
                gone.append(int(b.table[i, p]))
                table[i, p] = (-1, 1 << 30, -(1 << 31))[p % 3]
    for x in (b.k, b.v):
        if 0 in gone or 0 not in b.table:
            x[0] = float("nan")
        for p in gone:
            x[p] = float("nan")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ripe_paged_attn(b.q, b.k, b.v, table, ctx, row0, b.out[:b.rows], b.lse[:b.rows], max_ntok=max(b.new), window=window,
                    sinks=sinks, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0 and (gone or window > 100)
    o, lse = b.out[:b.rows].float().cpu().numpy(), b.lse[:b.rows].cpu().numpy()
    vmax = 6.0  # of that many normal deviates
    tol = 2 ** -8 * np.abs(ref) + (2 ** -8 + 2 ** -12) * vmax if b.dtype == torch.bfloat16 else 2e-5 * vmax
    assert (np.abs(o - ref) <= tol).all() and np.abs(lse - ref_lse).max() <= 2e-4


@pytest.mark.parametrize("d,page", [(128, 64), (96, 32), (64, 16)])
def test_both_row_tiles_of_an_item_know_of_values_that_are_not_finite(d, page):
    """Two row tiles over the same key tiles, each of whose values is not finite somewhere:
    whichever of the two softmax groups comes to a tile first, both give what the formula
    gives, every time."""
    from depth_planed_kv_b200.ripe import ripe_paged_attn
    b = Batch([40, 333, 7], [256, 250, 200], 4, 2, d, page, seed=44)
    for i in range(3):
        for pos in range(b.ctx[i], b.ctx[i] + b.new[i], 29):   # channel by channel, seen by later rows
            ch = pos * 5 % d
            b.v[int(b.table[i, pos // page]), pos % 2, pos % page, ch] = (float("nan"), float("inf"), -float("inf"))[pos % 3]
    ref, _ = b.oracle()
    dev = b.dev()
    ok = np.isfinite(ref)
    assert not ok.all() and ok.any()
    for _ in range(60):
        ripe_paged_attn(b.q, b.k, b.v, *dev, b.out[:b.rows], b.lse[:b.rows], max_ntok=max(b.new))
        got = b.out[:b.rows].float().cpu().numpy()
        assert (np.isnan(got) == np.isnan(ref)).all() and (np.isposinf(got) == np.isposinf(ref)).all()
        assert (np.isneginf(got) == np.isneginf(ref)).all() and np.abs(got[ok] - ref[ok]).max() < 0.05


def test_calls_without_an_error_word_report_to_the_devices_own():
    from depth_planed_kv_b200.ripe import ripe_paged_append, ripe_paged_attn, ripe_paged_get_device_error
    b = Batch([20, 30, 40], [2, 3, 1], 4, 2, 64, 16, seed=45)
    k = torch.randn((b.rows, 2, 64)).to(b.dtype).cuda()
    table, ctx, row0 = b.dev()
    assert ripe_paged_get_device_error() == 0
    ripe_paged_append(k, k, b.k, b.v, table, ctx, row0)
    ripe_paged_attn(b.q, b.k, b.v, table, ctx, row0, b.out[:b.rows], max_ntok=3)
    assert ripe_paged_get_device_error() == 0
    # a sequence longer than max_ntok: left as it was, and said so
    b.out.fill_(77.0)
    ripe_paged_attn(b.q, b.k, b.v, table, ctx, row0, b.out[:b.rows], max_ntok=2)
    assert ripe_paged_get_device_error("cuda") == 8 and ripe_paged_get_device_error() == 0
    assert bool((b.out[2:5] == 77.0).all()) and not bool((b.out[:2] == 77.0).any())
    for what, code in (("ctx", 2), ("descend", 8), ("page", 9)):
        dev, _, _ = bad_batch(b, what)
        ripe_paged_append(k, k, b.k, b.v, *dev)
        assert ripe_paged_get_device_error() == code
        ripe_paged_attn(b.q, b.k, b.v, *dev, b.out[:b.rows], max_ntok=30)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        assert ripe_paged_get_device_error(0, s) == code
    # the caller's word keeps what it is told apart
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ripe_paged_append(k, k, b.k, b.v, *dev, err=err)
    assert ripe_paged_get_device_error() == 0 and int(err) == 9


FIRST_IN_CAPTURE = """
import torch
from depth_planed_kv_b200.ripe import ripe_paged_append, ripe_paged_attn, ripe_paged_get_device_error, ripe_sample
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
p = torch.randn((4, 2, 16, 64), device="cuda").bfloat16()
k, q = torch.randn((3, 2, 64), device="cuda").bfloat16(), torch.randn((3, 4, 64), device="cuda").bfloat16()
o = torch.zeros_like(q)
table, ctx, row0 = i32([[1, 2], [3, 0]]), i32([14, 5]), i32([0, 2, 3])
z, u = torch.randn((3, 5000), device="cuda"), torch.rand(3, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    ripe_paged_append(k, k, p, p, table, ctx, row0)
    ripe_paged_attn(q, p, p, table, ctx, row0, o, max_ntok=2)
    tok, _ = ripe_sample(z, u)
g.replay()
assert ripe_paged_get_device_error() == 0
want = o.clone()
ripe_paged_attn(q, p, p, table, ctx, row0, o, max_ntok=2)
assert bool((o == want).all()) and bool((tok == ripe_sample(z, u)[0]).all())
row0.copy_(i32([0, 3, 3]))   # three tokens where max_ntok says two
g.replay()
assert ripe_paged_get_device_error() == 8
print("captured first")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("case", [([40], [6], 2, 2, 64, 16, "f32"), ([40], [6], 2, 2, 80, 32, "bf16"), ([40], [6], 2, 2, 64, 16, "bf16"),
                                  ([40], [60], 2, 2, 64, 16, "bf16")], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_value_that_is_seen_counts_however_small_its_weight(case, bad):
    """The weight of a key whose score is 300 below the largest is 0 in 32 bits; a NaN or
    infinity it carries still makes the row one that is not finite, and no other row."""
    from depth_planed_kv_b200.ripe import ripe_paged_attn
    b = Batch(*case, seed=46)
    pos = b.ctx[0] + 2
    at = int(b.table[0, pos // b.page]), slice(None), pos % b.page
    b.q[:] = 1.0
    b.k[at] = -300.0 / b.d ** 0.5   # score -300, beside normal ones
    b.v[at[0], :, at[2], 5] = bad
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ripe_paged_attn(b.q, b.k, b.v, *b.dev(), b.out[:b.rows], max_ntok=max(b.new), err=err)
    o = b.out[:b.rows].float().cpu().numpy()
    assert int(err) == 0
    assert np.isfinite(o[:2]).all() and not np.isfinite(o[2:, :, 5]).any()
    assert np.isfinite(np.delete(o, 5, axis=2)).all()


@pytest.mark.parametrize("new,dtype", [([1, 0, 2, 0], "bf16"), ([40, 0, 60, 0], "bf16"), ([3, 0, 30, 0], "f32")], ids=str)
@pytest.mark.parametrize("pad", [3, 500])
def test_a_padded_batchs_empty_sequences_may_hold_anything(new, dtype, pad):
    """Sequences without tokens, among the others and behind them, with lengths and pages that
    mean nothing, are neither served nor reported."""
    from depth_planed_kv_b200.ripe import ripe_paged_append, ripe_paged_attn
    b = Batch([20, 30, 40, 9], new, 4, 2, 64, 16, dtype, seed=47)
    ref, _ = b.oracle()
    table = torch.cat([b.table, torch.full((pad, b.table.shape[1]), -9, dtype=torch.int32)])
    table[1] = 1 << 30
    ctx = [20, -1, 40, (1 << 31) - 1] + [(-1, 1 << 30, -(1 << 31))[i % 3] for i in range(pad)]
    row0 = list(b.row0) + [b.rows] * pad
    dev = [torch.as_tensor(np.asarray(x, np.int32)).cuda() for x in (table.numpy(), ctx, row0)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k0 = b.k.clone()
    ripe_paged_attn(b.q, b.k, b.v, *dev, b.out[:b.rows], max_ntok=max(new), err=err)
    k = torch.randn((b.rows, 2, 64)).to(b.dtype).cuda()
    ripe_paged_append(k, k, b.k, b.v, *dev, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    assert np.abs(b.out[:b.rows].float().cpu().numpy() - ref).max() < 0.05
    assert int((b.k != k0).any(-1).sum()) == b.rows * 2


@pytest.mark.parametrize("nseq,new", [(3, 20), (40, 1), (600, 3)])
def test_descending_offsets_are_what_is_reported(nseq, new):
    """Not what they make of the sequences behind them, here more tokens than the pages hold."""
    from depth_planed_kv_b200.ripe import ripe_paged_append, ripe_paged_attn
    b = Batch([20] * nseq, [new] * nseq, 4, 2, 64, 16, seed=48)
    table, ctx, row0 = b.dev()
    row0[2] = row0[1] - 1
    row0[3:] = b.rows
    if nseq > 3:
        ctx[3:] = 1 << 29
        row0[3] = 0
    k = torch.randn((b.rows, 2, 64)).to(b.dtype).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(50):
        for max_ntok in (1 << 20, 4):
            ripe_paged_attn(b.q, b.k, b.v, table, ctx, row0, b.out[:b.rows], max_ntok=max(max_ntok, new), err=err)
            assert int(err) == 8
            err.zero_()
        ripe_paged_append(k, k, b.k, b.v, table, ctx, row0, err=err)
        assert int(err) == 8
        err.zero_()
