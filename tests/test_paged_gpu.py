"""The paged single-plane cache on the GPU (ripe_paged_append, ripe_paged_attn) against
the fp64 oracle, through the binding.

Tolerances, from the formats.  bf16 has 8 significant bits: eps = 2^-7, and a rounding
is off by at most half of that, 2^-8 of the value.  P is rounded once and O once; the
products are exact and the sums in fp32 (2^-24 each, over thousands of terms below
2^-12).  With sum p = 1 the first is at most 2^-8 * sum p|v| <= 2^-8 * max|v| of the row,
so |err| <= 2^-8 |o| + (2^-8 + 2^-12) max|v| (2^-12 also covers the product of the two);
max|v| is taken over all values that any row could see.  lse: scores are sums of d
products in fp32, error <= d * 2^-24 * sum|q k| scale; ex2 adds 2^-22 relative:
2e-4 absolute covers |q k| scale sums up to 100 at d = 128.  f32: sums of up to some
thousand terms in fp32: 2^-24 * (d + keys) * max|v| relative to the row, 2e-5 with the
sizes used here."""
import numpy as np
import pytest
import torch

from oracle import paged as PG

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Batch:
    """Random pages, table and rows for the given lengths; numpy copies beside the tensors."""

    def __init__(self, ctx, new, H, Hkv, d, page, dtype="bf16", token_major=False, seed=0, spare=5, pad_q=0, poison=None):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.new, self.H, self.Hkv, self.d, self.page = list(ctx), list(new), H, Hkv, d, page
        self.dtype = DT[dtype]
        need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
        npages = sum(need) + spare
        order = torch.randperm(npages, generator=g)
        shape = (npages, page, Hkv, d) if token_major else (npages, Hkv, page, d)
        def pool():
            x = torch.randn(shape, generator=g).to(self.dtype).cuda()
            return x.transpose(1, 2) if token_major else x
        self.k, self.v = pool(), pool()
        width = max(1, max(need))
        self.table = torch.full((len(need), width), -7, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n].to(torch.int32)
            at += n
        self.row0 = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.rows = int(self.row0[-1])
        if poison is not None:   # slots behind each sequence's last token, and the spare pages
            for i, n in enumerate(need):
                end = (ctx[i] + new[i]) % page
                if n and end:
                    for x in (self.k, self.v):
                        x[int(self.table[i, n - 1]), :, end:] = poison
            for p in order[at:]:
                self.k[int(p)] = poison
                self.v[int(p)] = poison
        store = torch.randn((self.rows, H + pad_q, d), generator=g).to(self.dtype).cuda()
        self.q = store[:, :H]
        self.out = torch.full((self.rows + 3, H, d), 77.0, dtype=self.dtype, device="cuda")
        self.lse = torch.full((self.rows + 3, H), 77.0, device="cuda")

    def dev(self):
        i32 = lambda x: torch.as_tensor(np.asarray(x, np.int32)).cuda()
        return self.table.cuda(), i32(self.ctx), i32(self.row0)

    def run(self, **kw):
        from depth_planed_kv_b200.ripe import ripe_paged_attn
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw.setdefault("max_ntok", max(1, max(self.new)))
        ripe_paged_attn(self.q, self.k, self.v, *self.dev(), self.out[:self.rows], self.lse[:self.rows], err=err, **kw)
        torch.cuda.synchronize()
        assert int(err) == 0
        # nothing behind the last row is touched
        assert bool((self.out[self.rows:] == 77.0).all()) and bool((self.lse[self.rows:] == 77.0).all())
        return self.out[:self.rows].float().cpu().numpy(), self.lse[:self.rows].cpu().numpy()

    def oracle(self, **kw):
        f = lambda x: x.float().cpu().numpy()
        return PG.attn(f(self.q), f(self.k), f(self.v), self.table.numpy(), self.ctx, self.row0, **kw)

    def check(self, **kw):
        got, got_lse = self.run(**kw)
        kw.pop("max_ntok", None)
        ref, ref_lse = self.oracle(**kw)
        finite = self.v.float()
        vmax = float(finite[torch.isfinite(finite)].abs().max())
        tol = 2 ** -8 * np.abs(ref) + (2 ** -8 + 2 ** -12) * vmax if self.dtype == torch.bfloat16 else 2e-5 * vmax
        assert (np.abs(got - ref) <= tol).all(), float(np.nanmax(np.abs(got - ref)))
        assert np.abs(got_lse - ref_lse).max() <= (2e-4 if self.dtype == torch.bfloat16 else 2e-5)
        # the largest error is far below those bounds unless something is off by a key
        rms = np.sqrt(np.mean(ref ** 2)) + 1e-9
        assert np.sqrt(np.mean((got - ref) ** 2)) / rms <= (4e-3 if self.dtype == torch.bfloat16 else 2e-6)


DECODE = [  # ctx, new, H, Hkv, d, page
    ([0], [1], 2, 2, 64, 16),
    ([1], [1], 1, 1, 128, 16),
    ([15, 16, 17, 63, 64, 65], [1] * 6, 4, 4, 96, 16),
    ([1024], [1], 55, 55, 96, 64),
    ([100, 0, 3000, 7], [1, 1, 1, 1], 16, 2, 128, 32),
    ([100, 200], [8, 8], 4, 4, 128, 128),
    ([511, 513, 40], [4, 1, 3], 8, 2, 64, 1024),
    ([33, 900], [2, 5], 9, 3, 96, 16),
    ([5000] * 3, [1] * 3, 32, 8, 128, 16),
    ([77], [16], 3, 3, 64, 64),
    ([40, 9], [1, 1], 14, 1, 128, 16),
]
CHUNK = [
    ([0], [17], 1, 1, 64, 16),
    ([0], [128], 2, 2, 128, 64),
    ([0], [129], 2, 2, 96, 32),
    ([0], [700], 3, 3, 64, 16),
    ([1000], [300], 8, 2, 128, 16),
    ([5, 0, 130, 1, 600], [40, 1, 0, 257, 64], 8, 4, 96, 128),
    ([2500], [33], 10, 2, 128, 64),
    ([300, 12], [40, 19], 15, 5, 64, 16),
    ([64], [9], 64, 1, 128, 256),
    ([900], [2], 100, 1, 64, 16),
    ([4000] * 4, [8] * 4, 32, 8, 128, 16),
    ([127, 128, 129], [129, 128, 127], 4, 4, 128, 128),
]
SIMT = [
    ([48], [4], 2, 2, 16, 16, "f32"),
    ([0], [1], 1, 1, 8, 16, "bf16"),
    ([100, 3], [1, 50], 6, 2, 80, 32, "bf16"),
    ([700, 0, 31], [3, 33, 1], 8, 1, 128, 64, "f32"),
    ([2000], [40], 4, 4, 64, 16, "f32"),
    ([5, 260], [17, 0], 16, 1, 32, 16, "f32"),
    ([90], [2], 3, 3, 4 * 5, 16, "f32"),
]


@pytest.mark.parametrize("case", DECODE, ids=str)
def test_decode_matches_oracle(case):
    Batch(*case, seed=1).check()


@pytest.mark.parametrize("case", CHUNK, ids=str)
def test_chunk_matches_oracle(case):
    Batch(*case, seed=2).check()


@pytest.mark.parametrize("case", SIMT, ids=str)
def test_cuda_core_form_matches_oracle(case):
    Batch(*case, seed=3).check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (64, 0), (100, 130), (257, 3), (5000, 9)])
@pytest.mark.parametrize("case", [DECODE[2], DECODE[4], DECODE[5], CHUNK[3], CHUNK[4], CHUNK[5], SIMT[2], SIMT[3]], ids=str)
def test_window_and_first_tokens(case, window, sinks):
    Batch(*case, seed=4).check(window=window, sinks=sinks)


@pytest.mark.parametrize("case", [DECODE[2], DECODE[4], CHUNK[4], CHUNK[5], SIMT[3]], ids=str)
def test_token_major_pages_and_strided_rows(case):
    Batch(*case, seed=5, token_major=True, pad_q=2).check(scale=0.3)


@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
@pytest.mark.parametrize("case", [DECODE[2], DECODE[4], DECODE[6], CHUNK[1], CHUNK[4], CHUNK[5], SIMT[2], SIMT[3]], ids=str)
def test_unused_slots_may_hold_anything(case, poison):
    Batch(*case, seed=6, poison=poison).check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("case", [([40, 300], [8, 8], 4, 2, 64, 16, "bf16"), ([300, 40], [60, 200], 4, 2, 128, 32, "bf16"),
                                  ([300, 40], [6, 20], 4, 2, 32, 16, "f32")], ids=str)
def test_hidden_values_do_not_matter_and_seen_ones_do(case, bad):
    """A new token's value that is not finite reaches the rows that see it and no other;
    a hidden key that is not finite reaches none."""
    b = Batch(*case, seed=7)
    i, j, ch = 1, b.new[1] // 2, 5
    pos = b.ctx[i] + j
    b.v[int(b.table[i, pos // b.page]), 1, pos % b.page, ch] = bad
    window = 24
    # a key far behind the window of every new token of sequence 0 (and not among the first)
    far = b.ctx[0] - window - 9
    if far > 2:
        b.k[int(b.table[0, far // b.page]), :, far % b.page] = bad
        b.v[int(b.table[0, far // b.page]), :, far % b.page] = bad
    got, lse = b.run(window=window, sinks=2)
    ref, ref_lse = b.oracle(window=window, sinks=2)
    assert np.isfinite(ref_lse).all() and np.abs(lse - ref_lse).max() < 2e-4
    assert (np.isnan(got) == np.isnan(ref)).all() and (np.isposinf(got) == np.isposinf(ref)).all()
    ok = np.isfinite(ref)
    assert np.isfinite(got[ok]).all() and not ok.all()
    assert np.abs(got[ok] - ref[ok]).max() < 0.05


def test_results_repeat_bit_for_bit_and_max_ntok_only_chooses_the_kernel():
    b = Batch([700, 3, 1500], [2, 1, 1], 8, 4, 128, 16, seed=8)
    o1, l1 = b.run()
    o2, l2 = b.run()
    assert (o1 == o2).all() and (l1 == l2).all()
    o3, l3 = b.run(max_ntok=64)      # the tensor-memory kernel
    assert np.abs(o3 - o1).max() < 0.03 and np.abs(l3 - l1).max() < 2e-4
    b.check(max_ntok=None)


def test_many_sequences():
    rng = np.random.default_rng(9)
    ctx = rng.integers(0, 60, 1024)
    Batch(ctx, [1] * 1024, 2, 1, 64, 16, seed=9).check()
    new = rng.integers(0, 3, 1024)
    Batch(ctx, new, 16, 1, 64, 16, seed=10).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("token_major", [False, True])
def test_append_matches_oracle_and_touches_nothing_else(dtype, token_major):
    from depth_planed_kv_b200.ripe import ripe_paged_append
    for ctx, new, Hkv, d, page in (([0], [1], 1, 8, 16), ([5, 0, 31, 64], [3, 0, 40, 1], 5, 96, 32),
                                   ([0, 100], [700, 28], 8, 128, 64), ([9] * 200, [1] * 200, 2, 64, 16)):
        b = Batch(ctx, new, Hkv, Hkv, d, page, dtype, token_major, seed=11)
        kv = torch.randn((b.rows, 3 * Hkv, d)).to(b.dtype).cuda()   # a fused projection's rows
        k, v = kv[:, Hkv:2 * Hkv], kv[:, 2 * Hkv:]
        rk, rv = b.k.float().cpu().numpy().copy(), b.v.float().cpu().numpy().copy()
        PG.append(k.float().cpu().numpy(), v.float().cpu().numpy(), rk, rv, b.table.numpy(), ctx, b.row0)
        ripe_paged_append(k, v, b.k, b.v, *b.dev())
        torch.cuda.synchronize()
        assert (b.k.float().cpu().numpy() == rk).all() and (b.v.float().cpu().numpy() == rv).all()


def test_sequences_that_do_not_fit_are_skipped():
    from depth_planed_kv_b200.ripe import ripe_paged_append, ripe_paged_attn
    for max_ntok, new in ((4, [2, 3, 1]), (60, [20, 60, 30])):
        b = Batch([20, 30, 40], new, 4, 2, 64, 16, seed=12)
        ref, _ = b.oracle()
        table, ctx, row0 = b.dev()
        for what, code in (("ctx", 2), ("neg", 2), ("rows", 8), ("page", 9)):
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            c, r, tb = ctx.clone(), row0.clone(), table.clone()
            if what == "ctx":
                c[1] = table.shape[1] * 16 - new[1] + 1
            elif what == "neg":
                c[1] = -1
            elif what == "rows":
                r[2] = r[1] - 1
            else:
                tb[1, 0] = b.k.shape[0]
            out = torch.full_like(b.out, 5.0)
            ripe_paged_attn(b.q, b.k, b.v, tb, c, r, out[:b.rows], max_ntok=max_ntok, err=err)
            torch.cuda.synchronize()
            assert int(err) == code, what
            o = out.float().cpu().numpy()
            a0, a1 = b.row0[1], b.row0[2]
            assert np.abs(o[:a0] - ref[:a0]).max() < 0.05
            if what in ("ctx", "neg"):
                assert (o[a0:a1] == 5.0).all() and np.abs(o[a1:b.rows] - ref[a1:]).max() < 0.05
            err.zero_()
            k0 = b.k.clone()
            k = torch.randn((b.rows, 2, 64)).to(b.dtype).cuda()
            if what != "rows":
                ripe_paged_append(k, k, k0, k0.clone(), tb, c, r, err=err)
                torch.cuda.synchronize()
                assert int(err) == (code if what != "page" else 0) or what == "page"


def test_captured_call_replays_with_new_lengths():
    from depth_planed_kv_b200.ripe import ripe_paged_append, ripe_paged_attn, ripe_paged_attn_workspace
    for new in ([1, 1], [9, 30]):
        b = Batch([300, 50], new, 8, 2, 128, 16, seed=13)
        table, ctx, row0 = b.dev()
        kn, vn = (torch.randn((b.rows, 2, 128)).to(b.dtype).cuda() for _ in range(2))
        work = torch.empty(ripe_paged_attn_workspace(b.k, 8, max(new)), dtype=torch.uint8, device="cuda")
        def step():
            ripe_paged_append(kn, vn, b.k, b.v, table, ctx, row0)
            ripe_paged_attn(b.q, b.k, b.v, table, ctx, row0, b.out[:b.rows], b.lse[:b.rows], max_ntok=max(new), work=work)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for c in ([300, 50], [17, 3], [299, 0]):
            ctx.copy_(torch.tensor(c, dtype=torch.int32))
            b.ctx = c
            graph.replay()
            torch.cuda.synchronize()
            got = b.out[:b.rows].float().cpu().numpy()
            ref, _ = b.oracle()
            assert np.abs(got - ref).max() < 0.05


def test_calls_on_two_streams_at_once():
    from depth_planed_kv_b200.ripe import ripe_paged_attn
    cases = [Batch([2000, 100], [40, 300], 8, 2, 128, 16, seed=14), Batch([900] * 20, [1] * 20, 8, 8, 96, 32, seed=15)]
    refs = [c.oracle()[0] for c in cases]
    devs = [c.dev() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, d, s in zip(cases, devs, streams):
            ripe_paged_attn(c.q, c.k, c.v, *d, c.out[:c.rows], max_ntok=max(c.new), stream=s)
    torch.cuda.synchronize()
    for c, r in zip(cases, refs):
        assert np.abs(c.out[:c.rows].float().cpu().numpy() - r).max() < 0.05


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 256])
def test_every_page_and_head_size_on_the_tensor_cores(page, d):
    """Tiles of one page and of several, whole and cut by a sequence's end inside a page; the
    slots behind it hold NaN."""
    b = Batch([700, 1, 131], [50, 70, 200], 6, 2, d, page, seed=16, poison=float("nan"), token_major=page == 32)
    b.check()
    b.check(window=90, sinks=20)


@pytest.mark.parametrize("case", [([9000], [6], 4, 2, 64, 16, "bf16"), ([9000], [60], 4, 2, 96, 16, "bf16"),
                                  ([9000, 5000], [70, 90], 6, 2, 128, 64, "bf16"), ([3000], [6], 4, 2, 32, 16, "f32")], ids=str)
def test_values_that_are_not_finite_in_an_item_cut_among_blocks(case):
    """As the test above, with contexts long enough that several blocks share the item."""
    b = Batch(*case, seed=17)
    for ch, bad in ((5, float("inf")), (9, float("nan")), (30, -float("inf"))):
        pos = b.ctx[0] + b.new[0] // 2
        b.v[int(b.table[0, pos // b.page]), 1, pos % b.page, ch] = bad
    got, lse = b.run()
    ref, ref_lse = b.oracle()
    assert np.abs(lse - ref_lse).max() < 2e-4
    assert (np.isnan(got) == np.isnan(ref)).all() and (np.isposinf(got) == np.isposinf(ref)).all()
    assert (np.isneginf(got) == np.isneginf(ref)).all()
    ok = np.isfinite(ref)
    assert not ok.all() and np.abs(got[ok] - ref[ok]).max() < 0.05


@pytest.mark.parametrize("dtype,new", [("bf16", [1, 2]), ("bf16", [60, 40]), ("f32", [3, 30])])
def test_pages_past_32_bit_offsets(dtype, new):
    """Pages whose first element lies past 2^32 elements of the pool; keys and values in one
    pool (the oracle gets the pages in use, renumbered)."""
    from depth_planed_kv_b200.ripe import ripe_paged_append, ripe_paged_attn
    npages, Hkv, page, d, H = 4200, 8, 1024, 128, 16
    assert (npages - 10) * Hkv * page * d > 1 << 32
    g = torch.Generator().manual_seed(18)
    pool = torch.empty((npages, Hkv, page, d), dtype=DT[dtype], device="cuda")
    ctx, used = [1500, 100], [npages - 1, npages - 3, npages - 4, 0]
    for p in used:
        pool[p] = torch.randn((Hkv, page, d), generator=g).to(DT[dtype]).cuda()
    table = np.array([[used[0], used[3]], [used[2], used[1]]], np.int32)
    small = np.array([[0, 3], [2, 1]])
    row0 = np.array([0, new[0], sum(new)], np.int32)
    kn, q = (torch.randn((sum(new), h, d), generator=g).to(DT[dtype]) for h in (Hkv, H))
    O = torch.empty((sum(new), H, d), dtype=DT[dtype], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.as_tensor(np.asarray(x, np.int32)).cuda()
    ripe_paged_append(kn.cuda(), kn.cuda(), pool, pool, i32(table), i32(ctx), i32(row0), err=err)
    ripe_paged_attn(q.cuda(), pool, pool, i32(table), i32(ctx), i32(row0), O, max_ntok=max(new), err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    few = torch.stack([pool[p] for p in used]).float().cpu().numpy()
    row = kn.float().numpy()
    for i in range(2):   # the write went where the table says
        for j in range(new[i]):
            pos = ctx[i] + j
            assert (few[small[i, pos // page], :, pos % page] == row[row0[i] + j]).all()
    ref, _ = PG.attn(q.float().numpy(), few, few, small, ctx, row0)
    got = O.float().cpu().numpy()
    vmax = np.abs(few).max()
    tol = 2 ** -8 * np.abs(ref) + (2 ** -8 + 2 ** -12) * vmax if dtype == "bf16" else 2e-5 * vmax
    assert (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("page", [16, 32, 64, 256])
def test_head_size_32_on_the_tensor_cores(page):
    """Few rows, and many, whole and cut; the slots behind a sequence's end hold NaN."""
    for ctx, new, H, Hkv in (([0, 15, 700, 64], [1, 1, 1, 1], 6, 2), ([900, 3], [3, 5], 3, 1), ([4000], [9], 16, 1),
                             ([700, 1, 131], [50, 70, 200], 6, 2), ([9000], [60], 4, 4)):
        b = Batch(ctx, new, H, Hkv, 32, page, seed=19, poison=float("nan"), token_major=page == 32)
        b.check()
        b.check(window=90, sinks=20)


@pytest.mark.parametrize("ctx,new,H", [([0], [130], 1), ([200], [20], 1), ([900], [260], 1), ([3000], [17], 2), ([6000], [40], 4),
                                       ([9000, 3], [20, 20], 1), ([250] * 40, [17] * 40, 1), ([63, 64, 65, 255, 257], [20] * 5, 3)])
def test_small_calls_cut_into_pieces(ctx, new, H):
    """One key/value head: less than half a block's least share each, items of one piece and of
    many, more blocks than a warp has lanes on one item; the same bits every time."""
    b = Batch(ctx, new, H, 1, 128, 64, seed=20)
    b.check()
    b.check(window=200, sinks=70)
    o1, l1 = b.run()
    o2, l2 = b.run()
    assert (o1 == o2).all() and (l1 == l2).all()
