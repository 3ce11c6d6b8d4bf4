"""Host-side refusals of the paged single-plane cache and the token draw (no GPU needed):
every argument error is found before anything is enqueued, with a status and a message."""
import ctypes
import struct

import pytest

OK, INVALID, CAPACITY, UNALIGNED, UNSUPPORTED = 0, 1, 2, 3, 7


def lib():
    from depth_planed_kv_b200 import build as B
    B.build()
    from depth_planed_kv_b200 import ripe
    return ripe


def pages(**kw):
    a = dict(K=1 << 20, V=1 << 21, ps=2 * 16 * 64, hs=16 * 64, js=64, npages=10, page=16, Hkv=2, d=64, dtype=0, r0=0, r1=0, r2=0)
    a.update(kw)
    return struct.pack("@PPqqq5i3i", *a.values())


def batch(**kw):
    a = dict(table=1 << 22, stride=4, ctx=1 << 23, row0=1 << 24, width=4, nseq=2, nrows=3, max_ntok=2, err=0)
    a.update(kw)
    return struct.pack("@PqPP4iP", *a.values())


def refused(rc, code):
    r = lib()
    assert rc == code, (rc, r._lib.ripe_last_error())
    assert code == OK or r._lib.ripe_last_error()


BAD_PAGES = [
    (dict(dtype=2), INVALID), (dict(Hkv=0), INVALID), (dict(Hkv=257), INVALID), (dict(d=256), UNSUPPORTED), (dict(d=4), UNSUPPORTED),
    (dict(d=20), UNALIGNED), (dict(page=24), INVALID), (dict(page=8), INVALID), (dict(page=2048), INVALID),
    (dict(npages=0), INVALID), (dict(js=32), INVALID), (dict(hs=0), INVALID), (dict(ps=-1), INVALID),
    (dict(js=68), UNALIGNED), (dict(r1=1), INVALID), (dict(K=0), INVALID), (dict(V=0), INVALID), (dict(K=(1 << 20) + 8), UNALIGNED),
]
BAD_BATCH = [
    (dict(nseq=-1), INVALID), (dict(nseq=1025), INVALID), (dict(nrows=-1), INVALID), (dict(width=0), INVALID),
    (dict(width=1 << 27, stride=1 << 27), INVALID), (dict(stride=3), INVALID), (dict(table=0), INVALID), (dict(ctx=0), INVALID),
    (dict(row0=0), INVALID), (dict(row0=(1 << 24) + 2), UNALIGNED), (dict(err=6), UNALIGNED),
]


@pytest.mark.parametrize("kw,code", BAD_PAGES, ids=str)
def test_bad_pages(kw, code):
    r = lib()
    refused(r._lib.ripe_paged_append(pages(**kw), batch(), 1 << 25, 1 << 25, 128, None), code)
    refused(r._lib.ripe_paged_attn(pages(**kw), batch(), 4, 1 << 25, 256, 0, 0, 0.0, 1 << 26, 256, None, 1 << 27, 1 << 30, None), code)


@pytest.mark.parametrize("kw,code", BAD_BATCH, ids=str)
def test_bad_batch(kw, code):
    r = lib()
    refused(r._lib.ripe_paged_append(pages(), batch(**kw), 1 << 25, 1 << 25, 128, None), code)
    refused(r._lib.ripe_paged_attn(pages(), batch(**kw), 4, 1 << 25, 256, 0, 0, 0.0, 1 << 26, 256, None, 1 << 27, 1 << 30, None), code)


def test_nothing_to_do_is_not_an_error():
    r = lib()
    for kw in (dict(nseq=0), dict(nrows=0)):
        refused(r._lib.ripe_paged_append(pages(), batch(**kw), None, None, 128, None), OK)
        refused(r._lib.ripe_paged_attn(pages(), batch(**kw), 4, None, 256, 0, 0, 0.0, None, 256, None, None, 0, None), OK)
    refused(r._lib.ripe_sample(0, 10, None, 1, 10, None, None, None, None, None, None, None, None), OK)


@pytest.mark.parametrize("k,v,stride,code", [(0, 1 << 25, 128, INVALID), (1 << 25, 0, 128, INVALID), (1 << 25, (1 << 25) + 4, 128, UNALIGNED),
                                             (1 << 25, 1 << 25, 127, INVALID), (1 << 25, 1 << 25, 132, UNALIGNED)])
def test_bad_rows(k, v, stride, code):
    refused(lib()._lib.ripe_paged_append(pages(), batch(), k, v, stride, None), code)


@pytest.mark.parametrize("window,sinks,scale", [(-1, 0, 0.0), (0, -1, 0.0), (0, 0, -1.0), (0, 0, float("nan")), (0, 0, float("inf"))])
def test_bad_settings(window, sinks, scale):
    refused(lib()._lib.ripe_paged_attn(pages(), batch(), 4, 1 << 25, 256, window, sinks, scale, 1 << 26, 256, None, 1 << 27,
                                       1 << 30, None), INVALID)


@pytest.mark.parametrize("H,ntok,kw,code", [(3, 1, {}, INVALID), (0, 1, {}, INVALID), (258, 1, {}, INVALID), (4, 0, {}, INVALID),
                                             (34, 1, dict(dtype=1), UNSUPPORTED), (34, 1, dict(d=32, js=64), UNSUPPORTED),
                                             (129, 1, dict(Hkv=1), UNSUPPORTED)])
def test_bad_heads(H, ntok, kw, code):
    out = ctypes.c_size_t()
    refused(lib()._lib.ripe_paged_attn_workspace(pages(**kw), H, ntok, ctypes.byref(out)), code)
    refused(lib()._lib.ripe_paged_attn_workspace(pages(**kw), 4, 1, None), INVALID)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), INVALID), (dict(n=(1 << 20) + 1), INVALID), (dict(V=0), INVALID), (dict(V=(1 << 23) + 1), INVALID),
    (dict(dtype=5), INVALID), (dict(stride=9), INVALID), (dict(z=None), INVALID), (dict(u=None), INVALID), (dict(token=None), INVALID),
    (dict(z=(1 << 20) + 2), UNALIGNED), (dict(u=(1 << 20) + 1), UNALIGNED), (dict(k=(1 << 20) + 2), UNALIGNED),
], ids=str)
def test_bad_draw(kw, code):
    a = dict(n=2, V=10, z=1 << 20, dtype=1, stride=10, u=1 << 20, t=None, k=None, p=None, m=None, token=1 << 21, lp=None)
    a.update(kw)
    refused(lib()._lib.ripe_sample(*a.values(), None), code)


def test_binding_checks_shapes_before_the_call():
    import torch
    r = lib()
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(AssertionError):   # host memory
        r._pages(k, k)
    assert r._PAGES.size == 72 and r._BATCH.size == 56


def test_reading_the_devices_error_word_wants_a_place_for_it():
    refused(lib()._lib.ripe_paged_get_device_error(None, None), INVALID)
