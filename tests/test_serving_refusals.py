"""What the entry points of verification, pages, slots and the latent cache refuse before any CUDA call (CPU only;
the pointers are never followed)."""
import ctypes

import pytest

from constrained_decoding_diffusion_gb300 import build, native

P = 0x10000  # a non-NULL, aligned address that no refused call follows


class Latent(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_void_p), ("format", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("latent_dim", ctypes.c_int32), ("rope_dim", ctypes.c_int32)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return native.load()


def latent(**kw):
    d = dict(rows=P, format=2, n_pages=4, page_size=16, latent_dim=256, rope_dim=32)
    d.update(kw)
    return Latent(**d)


def refused(lib, rc, code=native.FA_ERR_INVALID_ARG):
    assert rc == code, rc
    assert lib.fa_last_error()


@pytest.mark.parametrize("kw", [dict(dtype=3), dict(dtype=-1), dict(B=-1), dict(B=65536), dict(T=0), dict(T=1025), dict(V=0),
                                dict(V=2147483647), dict(target=None), dict(target=P + 2), dict(draft=P + 1),
                                dict(tokens=None), dict(parents=None), dict(u=None), dict(S=-1), dict(S=5000), dict(S=0),
                                dict(states=None), dict(live=None), dict(path=None), dict(kept=None), dict(token=None),
                                dict(state=None)])
def test_verify(lib, kw):
    a = dict(dtype=0, B=1, T=4, V=100, target=P, draft=P, tokens=P, parents=P, u=P, states=P, S=5, live=P, path=P, kept=P,
             token=P, state=P)
    a.update(kw)
    refused(lib, lib.fa_verify(a["dtype"], a["B"], a["T"], a["V"], a["target"], 400, 100, a["draft"], 400, 100, a["tokens"],
                               a["parents"], None, a["u"], a["states"], a["S"], P, a["live"], a["path"], a["kept"], a["token"],
                               a["state"], None))


@pytest.mark.parametrize("kw", [dict(B=-1), dict(B=65536), dict(per=-1), dict(size=0), dict(size=24), dict(size=2048),
                                dict(size=-16), dict(n=-1), dict(B=65535, per=65535), dict(want=None), dict(table=None),
                                dict(held=None), dict(free=None), dict(n_free=None), dict(status=None)])
def test_pages_resize(lib, kw):
    a = dict(B=2, per=8, size=16, n=10, want=P, table=P, held=P, free=P, n_free=P, status=P)
    a.update(kw)
    refused(lib, lib.fa_pages_resize(a["B"], a["per"], a["size"], a["n"], a["want"], a["table"], a["held"], a["free"],
                                     a["n_free"], a["status"], None))


@pytest.mark.parametrize("kw", [dict(B=-1), dict(B=65536), dict(N=-1), dict(size=0), dict(size=24), dict(size=2048),
                                dict(n=-1), dict(n=1 << 28), dict(per=-1), dict(table=None), dict(start=None),
                                dict(count=None), dict(slot=None)])
def test_slot_map(lib, kw):
    a = dict(B=2, N=5, size=16, n=10, table=P, per=8, start=P, count=P, slot=P)
    a.update(kw)
    refused(lib, lib.fa_slot_map(a["B"], a["N"], a["size"], a["n"], a["table"], a["per"], a["start"], a["count"], a["slot"], P, P,
                                 P, None))


def write(lib, c, dtype=0, N=1, x=P, key=P, slot=P, pos=None, phase=None, inter=0):
    return lib.fa_latent_write(c, dtype, N, x, 256, key, 32, slot, pos, phase, inter, 1.0, None)


def attend(lib, c, dtype=2, B=1, T=1, heads=4, q=P, stride=288, table=P, per=2, length=P, scale=1.0, out=P, wsp=P, ws=1 << 40):
    return lib.fa_latent_attention(c, dtype, B, T, heads, q, 288 * 4, stride, 288, table, per, length, None, None, scale, out,
                                   None, wsp, ws, None)


@pytest.mark.parametrize("kw", [dict(format=0), dict(format=3), dict(page_size=0), dict(page_size=24), dict(page_size=2048),
                                dict(latent_dim=64), dict(latent_dim=192), dict(latent_dim=640), dict(rope_dim=0),
                                dict(rope_dim=24), dict(rope_dim=80), dict(n_pages=-1), dict(n_pages=1 << 28), dict(rows=None),
                                dict(rows=P + 8)])
def test_caches(lib, kw):
    c = ctypes.byref(latent(**kw))
    refused(lib, write(lib, c))
    refused(lib, lib.fa_latent_keep(c, 1, 1, P, 2, P, P, None))
    refused(lib, attend(lib, c))


def test_latent_calls(lib):
    c = ctypes.byref(latent())
    refused(lib, write(lib, None))
    for kw in (dict(dtype=3), dict(N=-1), dict(x=None), dict(key=None), dict(slot=None), dict(pos=P), dict(phase=P), dict(inter=2)):
        refused(lib, write(lib, c, **kw))
    for B, n, table, per, length, path in ((-1, 1, P, 2, P, P), (1, -1, P, 2, P, P), (1, 1025, P, 2, P, P), (1, 1, None, 2, P, P),
                                           (1, 1, P, -1, P, P), (1, 1, P, 2, None, P), (1, 1, P, 2, P, None)):
        refused(lib, lib.fa_latent_keep(c, B, n, table, per, length, path, None))


@pytest.mark.parametrize("kw,code", [(dict(dtype=0), 5), (dict(dtype=1), 5), (dict(dtype=7), 5), (dict(B=-1), 1), (dict(B=70000), 1),
                                     (dict(T=-1), 1), (dict(T=1025), 1), (dict(heads=0), 1), (dict(heads=1025), 1),
                                     (dict(q=None), 1), (dict(q=P + 2), 1), (dict(stride=287), 1), (dict(length=None), 1),
                                     (dict(table=None), 1), (dict(per=1 << 28), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
                                     (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(out=None), 1),
                                     (dict(out=P + 8), 1), (dict(ws=0), 4), (dict(wsp=None), 4), (dict(wsp=P + 16), 1),
                                     (dict(B=65535, T=1024, heads=1024), 1), (dict(B=60000, T=1, heads=64, per=1 << 23), 1)])
def test_latent_attention(lib, kw, code):
    refused(lib, attend(lib, ctypes.byref(latent()), **kw), code)


def test_latent_attention_workspace(lib):
    n = ctypes.c_size_t()
    for a in ((1, 1, 4, 256, 32, None), (1, 1, 0, 256, 32, ctypes.byref(n)), (1, 1, 4, 200, 32, ctypes.byref(n)),
              (1, 1, 4, 256, 8, ctypes.byref(n)), (-1, 1, 4, 256, 32, ctypes.byref(n))):
        refused(lib, lib.fa_latent_attention_workspace_bytes(*a))
    assert lib.fa_latent_attention_workspace_bytes(16, 64, 32, 512, 64, ctypes.byref(n)) == native.FA_OK


def test_nothing_to_do(lib):
    """Empty batches are fine and launch nothing."""
    c = ctypes.byref(latent())
    none = ctypes.byref(latent(n_pages=0, rows=None))
    assert lib.fa_verify(0, 0, 4, 100, *[None] * 1, 0, 0, None, 0, 0, None, None, None, None, None, 0, None, None, None, None, None,
                         None, None) == native.FA_OK
    assert lib.fa_pages_resize(0, 8, 16, 10, None, None, None, None, None, None, None) == native.FA_OK
    assert lib.fa_slot_map(0, 0, 16, 10, None, 8, None, None, None, None, None, None, None) == native.FA_OK
    assert write(lib, c, N=0, x=None, key=None, slot=None) == native.FA_OK
    assert write(lib, none, N=0) == native.FA_OK
    assert lib.fa_latent_keep(c, 0, 4, P, 2, None, None, None) == native.FA_OK
    assert lib.fa_latent_keep(c, 4, 0, P, 2, None, None, None) == native.FA_OK
    assert attend(lib, c, B=0, q=None, out=None, length=None, ws=0) == native.FA_OK
    assert attend(lib, c, T=0, q=None, out=None, length=None, ws=0) == native.FA_OK
