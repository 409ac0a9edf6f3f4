"""Refusals of the 8-bit cache entry points, before anything is launched (no
GPU: pointers are never followed)."""
import ctypes as C

import pytest

OK, INVALID, MISALIGNED, UNSUPPORTED, NOT_INIT = 0, 1, 2, 3, 4
A, BAD = 0x10000, 0x10008


@pytest.fixture(scope="module")
def fs():
    from rank_transformer_b200 import build
    build.build()
    from rank_transformer_b200 import flashsvd
    return flashsvd


def _cache(fs, **kw):
    f = dict(format=0, B=1, H_kv=2, D=64, S_max=128, k=A, v=A, k_scale=A, v_scale=A, k_tail=A, v_tail=A)
    f.update(kw)
    return fs.Kv8(*(f[n] for n, _ in fs.Kv8._fields_))


BAD_CACHES = [
    (dict(format=2), INVALID), (dict(format=-1), INVALID), (dict(B=-1), INVALID), (dict(H_kv=0), INVALID),
    (dict(S_max=0), INVALID), (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED),
    (dict(S_max=100), UNSUPPORTED), (dict(B=40000), UNSUPPORTED), (dict(k=None), INVALID),
    (dict(v_tail=None), INVALID), (dict(k_scale=BAD), MISALIGNED), (dict(v=BAD), MISALIGNED),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_cache(fs, kw, status):
    c = _cache(fs, **kw)
    assert fs.lib.flashsvd_kv8_store(A, A, C.byref(c), None, 64, 64, None) == status


def test_store_refusals(fs):
    c = _cache(fs)
    f = fs.lib.flashsvd_kv8_store
    assert f(A, A, None, None, 64, 64, None) == INVALID
    assert f(None, A, c, None, 64, 64, None) == INVALID
    assert f(A, BAD, c, None, 64, 64, None) == MISALIGNED
    assert f(A, A, c, None, -1, 64, None) == INVALID
    assert f(A, A, c, None, 64, 63, None) == INVALID
    assert f(A, A, c, None, 129, 129, None) == INVALID
    assert f(A, A, c, None, 0, 0, None) == OK
    assert f(A, A, _cache(fs, B=0), None, 64, 64, None) == OK


def test_need_init(fs):
    c = _cache(fs)
    L = fs.lib
    if L.flashsvd_lowrank_linear(A, A, A, None, A, 1, 64, 64, 64, None) != NOT_INIT:
        pytest.skip("library already initialised in this process")
    assert L.flashsvd_kv8_decode_attn(A, A, A, c, A, None, 0, A, 2, 1.0, None) == NOT_INIT
    assert L.flashsvd_attn_weight_sums(A, A, A, None, 1, 8, 2, 2, 64, 8, 8, 8, 1.0, None) == NOT_INIT
    assert L.flashsvd_kv8_evict(c, c, A, A, A, A, A, 64, 0, None) == NOT_INIT


def test_handle_checks(fs):
    """KV8Cache takes only tensors of its layout."""
    torch = pytest.importorskip("torch")
    from rank_transformer_b200.kv8 import KV8Cache
    c = KV8Cache(2, 3, 64, 128, "e4m3", device="cpu")
    assert (c.fmt, c.B, c.H_kv, c.D, c.S_max) == ("e4m3", 2, 3, 64, 128)
    assert c.struct.format == fs.KV8_E4M3 and c.struct.k == c.k.data_ptr()
    assert c.bytes() == 2 * (2 * 3 * 128 * 64 + 2 * 3 * 2 * 4 + 2 * 3 * 64 * 64 * 2)
    for i, t in enumerate((c.k.float(), c.v.transpose(0, 1), c.k_scale.double(), c.v_scale[:, :, :1],
                           c.k_tail.float(), c.v_tail.permute(0, 1, 3, 2))):
        args = list(c.tensors())
        args[i] = t
        with pytest.raises(ValueError):
            KV8Cache.from_tensors(*args)
    with pytest.raises(ValueError):
        KV8Cache(1, 1, 64, 100, device="cpu")
    with pytest.raises(ValueError):
        KV8Cache(1, 1, 64, 128, "int4", device="cpu")
