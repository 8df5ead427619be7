"""What the model-side entry points refuse before any CUDA call: sizes, types, formats, missing
buffers (CPU only; the pointers are never followed)."""
import ctypes

import pytest

from constrained_decoding_diffusion_gb300 import build, native

P = 0x10000  # a non-NULL, aligned address that no refused call follows


class Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("format", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return native.load()


def cache(**kw):
    d = dict(k=P, v=P, k_scale=P, v_scale=P, format=3, n_pages=4, page_size=16, kv_heads=2, head_dim=64)
    d.update(kw)
    return Cache(**d)


def refused(lib, rc, code=native.FA_ERR_INVALID_ARG):
    assert rc == code, rc
    assert lib.fa_last_error()


@pytest.mark.parametrize("kw", [dict(dtype=3), dict(dtype=-1), dict(n=-1), dict(dim=0), dict(dim=2000), dict(rot=3),
                                dict(rot=66), dict(rot=-2), dict(inter=2), dict(pos=None), dict(phase=None), dict(x=None),
                                dict(out=None)])
def test_rope(lib, kw):
    a = dict(dtype=0, n=4, heads=2, dim=64, rot=64, inter=0, x=P, pos=P, phase=P, out=P)
    a.update(kw)
    refused(lib, lib.fa_rope(a["dtype"], a["n"], a["heads"], a["dim"], a["rot"], a["inter"], 0, a["x"], 128, 64, a["pos"],
                             a["phase"], 1.0, a["out"], 128, 64, None))


BAD_CACHES = [dict(format=0), dict(format=4), dict(page_size=0), dict(page_size=24), dict(page_size=2048), dict(head_dim=8),
              dict(head_dim=72), dict(head_dim=272), dict(kv_heads=0), dict(n_pages=-1), dict(k=None), dict(v=P + 8),
              dict(k_scale=None), dict(v_scale=None)]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_caches(lib, kw):
    c = ctypes.byref(cache(**kw))
    refused(lib, lib.fa_cache_write(c, 0, 1, 1, P, 64, 64, 64, P, 64, 64, 64, P, 2, P, None, None, None, 0, 0, 1.0, None))
    refused(lib, lib.fa_cache_read(c, 0, 1, 1, P, 2, P, P, P, None))
    refused(lib, lib.fa_cache_keep(c, 1, 1, P, 2, P, P, None))
    refused(lib, lib.fa_tree_attention(c, 1, 1, 1, 2, P, 64, 64, 64, P, 2, P, None, None, 1.0, P, None, P, 1 << 40, None))


def test_cache_calls(lib):
    c = ctypes.byref(cache())
    refused(lib, lib.fa_cache_write(None, 0, 1, 1, P, 64, 64, 64, P, 64, 64, 64, P, 2, P, None, None, None, 0, 0, 1.0, None))
    for B, T, start, pos, phase, rot in ((-1, 1, P, None, None, 0), (1, -1, P, None, None, 0), (1, 1, None, None, None, 0),
                                         (1, 1, P, P, None, 16), (1, 1, P, None, P, 16), (1, 1, P, P, P, 15),
                                         (1, 1, P, P, P, 80)):
        refused(lib, lib.fa_cache_write(c, 0, B, T, P, 64, 64, 64, P, 64, 64, 64, P, 2, start, None, pos, phase, rot, 0, 1.0, None))
    refused(lib, lib.fa_cache_write(c, 5, 1, 1, P, 64, 64, 64, P, 64, 64, 64, P, 2, P, None, None, None, 0, 0, 1.0, None))
    refused(lib, lib.fa_cache_read(c, 0, 1, 1, P, 2, P, P, P + 4, None))
    refused(lib, lib.fa_cache_read(c, 0, 1, 1, None, 2, P, P, P, None))
    refused(lib, lib.fa_cache_read(c, 0, 1, 1, P, -1, P, P, P, None))
    refused(lib, lib.fa_cache_keep(c, 1, 1, P, 2, P, None, None))
    refused(lib, lib.fa_tree_mask(1, 1025, P, P, None, None))
    refused(lib, lib.fa_tree_mask(1, 5, P, None, None, None))


@pytest.mark.parametrize("kw,code", [(dict(dtype=0), 5), (dict(dtype=7), 5), (dict(heads=3), 1), (dict(T=-1), 1),
                                     (dict(T=1025), 1), (dict(B=70000), 1), (dict(q=None), 1), (dict(q=P + 2), 1),
                                     (dict(stride=63), 1), (dict(length=None), 1), (dict(out=None), 1), (dict(ws=0), 4),
                                     (dict(wsp=P + 16), 1), (dict(fmt=1, dtype=2), 5), (dict(head_dim=144), 5)])
def test_tree_attention(lib, kw, code):
    a = dict(dtype=1, B=1, T=1, heads=2, q=P, stride=64, length=P, out=P, ws=1 << 40, wsp=P, fmt=3, head_dim=64)
    a.update(kw)
    c = cache(format=a["fmt"], head_dim=a["head_dim"])
    refused(lib, lib.fa_tree_attention(ctypes.byref(c), a["dtype"], a["B"], a["T"], a["heads"], a["q"], 64, a["stride"], 64, P, 2,
                                       a["length"], None, None, 1.0, a["out"], None, a["wsp"], a["ws"], None), code)


def test_tree_attention_workspace(lib):
    n = ctypes.c_size_t()
    refused(lib, lib.fa_tree_attention_workspace_bytes(1, 1, 4, 2, 64, None))
    refused(lib, lib.fa_tree_attention_workspace_bytes(1, 1, 4, 0, 64, ctypes.byref(n)))
    refused(lib, lib.fa_tree_attention_workspace_bytes(1, 1, 5, 2, 64, ctypes.byref(n)))
    refused(lib, lib.fa_tree_attention_workspace_bytes(1, 1, 4, 2, 256, ctypes.byref(n)), native.FA_ERR_UNSUPPORTED)
    assert lib.fa_tree_attention_workspace_bytes(16, 64, 32, 8, 128, ctypes.byref(n)) == native.FA_OK


@pytest.mark.parametrize("kw,code", [(dict(dtype=4), 1), (dict(N=-1), 1), (dict(K=0), 1), (dict(V=0), 1),
                                     (dict(K=1 << 16, V=1 << 16), 1), (dict(top=0), 1), (dict(top=257), 1), (dict(S=-1), 1),
                                     (dict(S=5000), 1), (dict(states=None), 1), (dict(live=None), 1), (dict(S=0), 1),
                                     (dict(logp=None), 1), (dict(logp=P + 2), 1), (dict(scores=None), 1), (dict(ws=8), 4),
                                     (dict(wsp=P + 8), 1)])
def test_beam_select(lib, kw, code):
    a = dict(dtype=0, N=1, K=4, V=100, top=4, logp=P, scores=P, S=5, states=P, live=P, ws=1 << 30, wsp=P)
    a.update(kw)
    refused(lib, lib.fa_beam_select(a["dtype"], a["N"], a["K"], a["V"], a["top"], a["logp"], 400, 100, a["scores"], a["states"],
                                    a["S"], P, a["live"], P, P, P, P, a["wsp"], a["ws"], None), code)


def test_beam_others(lib):
    n = ctypes.c_size_t()
    refused(lib, lib.fa_beam_select_workspace_bytes(1, 4, 100, 300, ctypes.byref(n)))
    refused(lib, lib.fa_beam_select_workspace_bytes(1, 4, 100, 4, None))
    refused(lib, lib.fa_beam_tables(None, P, P, None))
    refused(lib, lib.fa_beam_reorder(1, 4, 4, 8, P, P, P, 8, P, None))
    refused(lib, lib.fa_beam_reorder(1, 4, 4, 8, P, None, P, 1, P, None))
    refused(lib, lib.fa_beam_reorder(1, 4, 4, -1, P, P, None, 0, P, None))


def test_nothing_to_do(lib):
    """Empty batches are fine and launch nothing."""
    c = ctypes.byref(cache())
    assert lib.fa_rope(0, 0, 2, 64, 64, 0, 0, None, 0, 0, P, P, 1.0, None, 0, 0, None) == native.FA_OK
    assert lib.fa_cache_write(c, 0, 0, 4, None, 0, 0, 0, None, 0, 0, 0, P, 2, None, None, None, None, 0, 0, 1.0, None) == native.FA_OK
    assert lib.fa_cache_read(c, 0, 4, 0, P, 2, None, None, None, None) == native.FA_OK
    assert lib.fa_tree_attention(c, 1, 4, 0, 2, None, 0, 0, 0, P, 2, None, None, None, 1.0, None, None, None, 0, None) == native.FA_OK
    assert lib.fa_beam_reorder(0, 4, 4, 8, None, None, None, 0, None, None) == native.FA_OK
