"""Pins of the plain cache model that the GPU tests compare with, and the host-side
refusals of the cache calls (CPU only)."""
import ctypes

import numpy as np
import torch

from compressed_sparse_attention_compress_gb300 import api
from tests import cache_helpers as ch


def test_codes_are_torchs_e4m3():
    rng = np.random.default_rng(0)
    x = np.clip(rng.standard_normal(20000) * np.exp(3 * rng.standard_normal(20000)), -448, 448).astype(np.float32)
    mid = ((ch.VALUES[:0x7E] + ch.VALUES[1:0x7F]) / 2).astype(np.float32)      # ties
    for v in (x, mid, -mid, np.array([-0.0, 0.0, 448.0], np.float32)):
        ref = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        np.testing.assert_array_equal(ch.e4m3_codes(v), ref)
    np.testing.assert_array_equal(ch.VALUES, torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double())


def test_block_scale():
    for v, s in [(448.0, 1.0), (448.1, 2.0), (0.0, 2.0 ** -126), (1.0, 2.0 ** -8), (np.inf, 2.0 ** -126)]:
        assert ch.block_scale(np.array([v, -0.0])) == s


def test_appending_rescales_earlier_codes():
    m = ch.Model(np.zeros((1, 1, 16, 64), np.uint8), np.ones((1, 1)), np.zeros((1, 1), np.int32))
    m.write(np.full((1, 1, 64), 1.0), [0, 1], [0])
    m.write(np.full((1, 1, 64), 1000.0), [0, 1], [1])
    rows = m.rows(0, [0, 1])
    assert rows[0, 0, 0] == 1.0 and rows[1, 0, 0] == 1024.0 and m.scale[0, 0] == 4.0


def test_attention_model_is_torchs():
    s = ch.Setup(0, 1, [40], 2, 64, 16, False, device="cpu")
    k, v = s.models()
    q = np.random.default_rng(1).standard_normal((1, 4, 64))
    out, lse, *_ = ch.attend(q, [0, 1], [39], 0.125, raw=(k, v), window=100)
    K, V = (torch.from_numpy(m.rows(0, range(40))).repeat_interleave(2, 1).transpose(0, 1) for m in (k, v))
    ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q).transpose(0, 1), K, V)
    np.testing.assert_allclose(out[0], ref[:, 0], rtol=1e-10, atol=1e-12)


P = ctypes.c_void_p
FAKE = 1 << 20      # an aligned address that the host checks alone look at


def _struct(**kw):
    s = api._CacheStruct()
    for k, v in dict(dict(k=FAKE, k_scale=FAKE, table=FAKE, n_blocks=4, max_blocks=2, block=16, H_kv=1, d=64),
                     **kw).items():
        setattr(s, k, v)
    return s


class _Handle(ctypes.Structure):
    """Room for a handle: the refusals below return before anything in it is used."""
    _fields_ = [("words", ctypes.c_int64 * 8)]


def _write(c, xk=FAKE, xv=None, B=1, T=4, dtype=0, cu=FAKE, pos0=FAKE):
    h = _Handle()
    return api.LIB.csa_cache_write(ctypes.addressof(h), ctypes.addressof(c), xk, xv, cu, pos0, B, T, dtype, None)


def _attn(cmp=None, raw=None, q=FAKE, idx=None, k_pad=0, cu_cmp=None, B=1, T=4, H=4, d=64, ratio=0, window=0, dtype=0,
          out=FAKE, ws=None, n=0):
    h = _Handle()
    a = [ctypes.addressof(c) if c is not None else None for c in (cmp, raw)]
    return api.LIB.csa_cache_attn_fwd(ctypes.addressof(h), q, a[0], a[1], idx, k_pad, cu_cmp, None, FAKE, FAKE, B, T, H,
                                      d, ratio, window, 0.1, dtype, out, None, ws, n, None)


def test_host_refusals_of_the_cache():
    assert _write(_struct(k=None)) == -1
    assert _write(_struct(k=FAKE + 8)) == -1
    assert _write(_struct(table=None)) == -1
    assert _write(_struct(v=FAKE)) == -1                      # V without its scales
    assert _write(_struct(v=FAKE, v_scale=FAKE)) == -1        # and without rows for it
    assert _write(_struct(), xv=FAKE) == -1
    assert _write(_struct(), xk=FAKE + 2) == -1
    assert _write(_struct(H_kv=0)) == -1
    assert _write(_struct(block=8)) == -2
    assert _write(_struct(block=48)) == -2
    assert _write(_struct(block=256)) == -2
    assert _write(_struct(d=32)) == -2
    assert _write(_struct(max_blocks=1 << 28)) == -2          # positions past 31 bits
    assert _write(_struct(), dtype=2) == -1
    assert _write(_struct(), B=-1) == -1
    assert _write(_struct(), cu=None) == -1


def test_host_refusals_of_the_attention():
    c = _struct()
    assert _attn() == -1                                      # no cache
    assert _attn(raw=c) == -1                                 # no window
    assert _attn(cmp=c) == -1                                 # no ratio
    assert _attn(raw=c, window=4, idx=FAKE, k_pad=4) == -1    # a list without compressed entries
    assert _attn(cmp=c, ratio=4, idx=FAKE, k_pad=0) == -1
    assert _attn(cmp=c, ratio=4, cu_cmp=FAKE) == -1
    assert _attn(raw=c, window=4, d=128) == -1
    assert _attn(raw=_struct(H_kv=3), window=4) == -1         # 4 heads over 3
    assert _attn(raw=c, window=4, H=129) == -2
    assert _attn(raw=c, window=4, q=FAKE + 4) == -1
    assert _attn(cmp=_struct(v=FAKE, v_scale=FAKE), raw=c, ratio=4, window=4) == -1
    assert _attn(cmp=_struct(H_kv=2), raw=c, ratio=4, window=4) == -1
    assert _attn(raw=c, window=4, dtype=7) == -1
    assert api.LIB.csa_cache_attn_workspace(None, 4, 4, 1, 64) == 0


def test_host_refusals_of_sizes():
    assert _write(_struct(H_kv=65537, n_blocks=1)) == -2
    assert _write(_struct(H_kv=65536, n_blocks=1), B=20000, T=1 << 20) == -2   # 105,536 blocks x 65,536 heads
    assert _attn(raw=_struct(H_kv=65537, n_blocks=1), window=4, H=65537) == -2


def test_python_checks():
    import pytest
    with pytest.raises(ValueError):
        api.Cache(torch.zeros(2, 1, 16, 64, dtype=torch.uint8), torch.ones(2, 1), torch.zeros(1, 1, dtype=torch.int32))
