"""csa_cache_write and csa_cache_read against the plain model: codes, scales and rows bit for bit."""
import numpy as np
import pytest
import torch

from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from compressed_sparse_attention_compress_gb300 import api  # noqa: E402


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rows(rng, T, H_kv, d, fp32, spread=1.0):
    x = rng.standard_normal((T, H_kv, d)) * np.exp(spread * rng.standard_normal((T, H_kv, 1)))
    t = torch.from_numpy(x.astype(np.float32)).to("cuda")
    return t if fp32 else t.to(torch.bfloat16)


def _same(cache, models):
    torch.cuda.synchronize()
    for m, (c, s) in zip(models, [(cache.k, cache.k_scale), (cache.v, cache.v_scale)]):
        if c is None:
            continue
        np.testing.assert_array_equal(s.cpu().numpy().astype(np.float64), m.scale)
        got = c.cpu().numpy()
        nan = (m.codes & 0x7F) == 0x7F
        np.testing.assert_array_equal((got & 0x7F) == 0x7F, nan)
        np.testing.assert_array_equal(got[~nan], m.codes[~nan])


CASES = [
    # lengths, first positions, H_kv, d, block, shared, fp32
    ([1, 1, 1], [0, 63, 64], 1, 128, 64, True, False),
    ([1] * 70, list(range(70)), 2, 64, 16, False, True),
    ([200, 0, 1, 17, 130], [5, 3, 127, 128, 0], 3, 128, 128, False, False),
    ([3, 500, 33], [31, 1, 0], 1, 64, 32, False, True),
    ([65, 64, 63], [0, 64, 1], 8, 128, 64, True, False),
    ([2, 3, 2, 4], [15, 14, 16, 13], 5, 64, 16, True, False),
]


@pytest.mark.parametrize("case", CASES)
def test_written_codes_scales_and_rows_read_back(case):
    n, pos0, H_kv, d, block, shared, fp32 = case
    B = len(n)
    s = ch.Setup(1, B, [p + m for p, m in zip(pos0, n)], H_kv, d, block, shared)
    h, cache, models = api.Handle(0), None, s.models()
    cache = api.Cache(**s.tensors())
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    T = int(cu[-1]) + 9                                   # capacity rows behind the last sequence
    xk, xv = _rows(s.rng, T, H_kv, d, fp32), _rows(s.rng, T, H_kv, d, fp32, 3.0)
    api.csa_cache_write(h, cache, xk, _i32(cu.tolist()), _i32(pos0), x_v=None if shared else xv)
    for m, x in zip(models if not shared else models[:1], [xk, xv]):
        m.write(x.float().cpu().numpy(), cu, pos0)
    _same(cache, models)
    # read back: exact in both types (a code has 4 significant bits)
    for dt in (torch.bfloat16, torch.float32):
        ko = torch.full((T, H_kv, d), 7.0, dtype=dt, device="cuda")
        vo = None if shared else torch.full_like(ko, 7.0)
        api.csa_cache_read(h, cache, _i32(cu.tolist()), _i32(pos0), ko, v_out=vo)
        torch.cuda.synchronize()
        for m, o in zip(models, [ko, vo]):
            if o is None:
                continue
            o = o.double().cpu().numpy()
            for b in range(B):
                np.testing.assert_array_equal(o[cu[b]:cu[b + 1]], m.rows(b, np.arange(pos0[b], pos0[b] + n[b])))
            assert not o[cu[-1]:].any()                   # capacity rows are zeros
    assert h.device_status() == 0


def test_token_by_token_equals_the_model_and_scales_only_grow():
    H_kv, d, block, steps = 2, 64, 16, 40
    s = ch.Setup(2, 2, [steps + 3, steps], H_kv, d, block, False)
    h, cache, models = api.Handle(0), api.Cache(**s.tensors()), s.models()
    cu = np.array([0, 1, 2], np.int32)
    for i in range(steps):
        pos = [i + 3, i]
        xk, xv = _rows(s.rng, 2, H_kv, d, False, 4.0), _rows(s.rng, 2, H_kv, d, False, 4.0)
        api.csa_cache_write(h, cache, xk, _i32(cu.tolist()), _i32(pos), x_v=xv)
        for m, x in zip(models, [xk, xv]):
            m.write(x.float().cpu().numpy(), cu, pos)
    _same(cache, models)
    assert h.device_status() == 0


def test_zero_tiny_huge_and_non_finite_rows():
    d, block = 64, 16
    s = ch.Setup(3, 1, [64], 1, d, block, True)
    h, cache, (m, _) = api.Handle(0), api.Cache(**s.tensors()), s.models()
    x = np.zeros((64, 1, d), np.float32)
    x[1] = 1e-30                                     # a zero row, then a tiny one in the same block
    x[5, 0, :4] = [-0.0, 0.0, 2.0 ** -149, -(2.0 ** -140)]
    x[16] = 3.3e38                                   # near the top of float32
    x[17, 0, 1] = -3.4e38
    x[32, 0, :3] = [np.nan, np.inf, -np.inf]         # beside ordinary values
    x[33] = s.rng.standard_normal(d)
    x[48:] = np.inf                                  # nothing finite in the block
    t = torch.from_numpy(x).cuda()
    api.csa_cache_write(h, cache, t, _i32([0, 64]), _i32([0]))
    m.write(x, [0, 64], [0])
    _same(cache, (m, m))
    # then a larger row joins a block that held zeros only so far
    y = np.full((1, 1, d), 0.75, np.float32)
    api.csa_cache_write(h, cache, torch.zeros(2, 1, d, device="cuda"), _i32([0, 2]), _i32([0]))
    api.csa_cache_write(h, cache, torch.from_numpy(y).cuda(), _i32([0, 1]), _i32([2]))
    m.write(np.zeros((2, 1, d)), [0, 2], [0])
    m.write(y, [0, 1], [2])
    _same(cache, (m, m))
    assert h.device_status() == 0


def test_scale_border_is_exact():
    # maxima at, just above and just below 448 * 2^e
    d, block = 64, 16
    s = ch.Setup(4, 6, [16] * 6, 1, d, block, True)
    h, cache, (m, _) = api.Handle(0), api.Cache(**s.tensors()), s.models()
    x = np.zeros((6 * 16, 1, d), np.float32)
    for b, v in enumerate([448.0, np.nextafter(np.float32(448), np.float32(1e9)),
                           np.nextafter(np.float32(448), np.float32(0)), 1.75, 448.0 * 2.0 ** -126, 2.0 ** -118]):
        x[16 * b, 0, 3] = v
    cu = np.arange(0, 97, 16).astype(np.int32)
    api.csa_cache_write(h, cache, torch.from_numpy(x).cuda(), _i32(cu.tolist()), _i32([0] * 6))
    m.write(x, cu, [0] * 6)
    _same(cache, (m, m))


def test_bad_positions_and_blocks_are_skipped_with_a_status():
    d, block, B = 64, 16, 4
    s = ch.Setup(5, B, [32] * B, 1, d, block, True)
    s.t_table[1, 1] = s.n                            # a block number out of range
    h, cache, (m, _) = api.Handle(0), api.Cache(**s.tensors()), s.models()
    before = cache.k.clone()
    x = _rows(s.rng, 4 * 20, 1, d, False)
    cu, pos0 = [0, 20, 40, 60, 80], [-1, 0, 13, 12]  # negative; bad second block; past the table; good
    api.csa_cache_write(h, cache, x, _i32(cu), _i32(pos0))
    assert h.device_status() == -6
    xs = x.float().cpu().numpy()
    ok = ch.Model(m.codes, m.scale, s.table[3:])
    ok.write(xs[60:], [0, 20], [12])
    got = cache.k.cpu().numpy()
    blocks = s.table[3]
    np.testing.assert_array_equal(got[blocks], ok.codes[blocks])
    np.testing.assert_array_equal(got[s.table[0]], before.cpu().numpy()[s.table[0]])
    np.testing.assert_array_equal(got[s.table[2]], before.cpu().numpy()[s.table[2]])
    o = torch.full((80, 1, d), 3.0, device="cuda")
    api.csa_cache_read(h, cache, _i32(cu), _i32(pos0), o)
    assert h.device_status() == -6
    assert not o[:20].any() and not o[36:60].any() and o[60:].any()


def test_refusals():
    h = api.Handle(0)
    s = ch.Setup(6, 1, [16], 2, 64, 16, False)
    t = s.tensors()
    cache = api.Cache(**t)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu, p0 = _i32([0, 4]), _i32([0])
    with pytest.raises(api.CSAError) as e:           # a cache with V takes both
        api.csa_cache_write(h, cache, x, cu, p0)
    assert e.value.code == -1
    with pytest.raises(ValueError):
        api.csa_cache_write(h, cache, x.transpose(0, 1).reshape(4, 2, 64)[:, :1], cu, p0, x_v=x)
    with pytest.raises(TypeError):
        api.csa_cache_write(h, cache, x.half(), cu, p0, x_v=x.half())
    with pytest.raises(TypeError):
        api.csa_cache_write(h, cache, x, cu.long(), p0, x_v=x)
    with pytest.raises(ValueError):                  # more sequences than tables
        api.csa_cache_write(h, cache, x, _i32([0, 2, 4]), _i32([0, 0]), x_v=x)
    with pytest.raises(ValueError):
        api.Cache(t["k"], t["k_scale"], t["table"], v=t["v"])
    with pytest.raises(ValueError):
        api.Cache(t["k"].transpose(0, 1), t["k_scale"], t["table"])
    odd = api.Cache(torch.zeros(2, 1, 24, 64, dtype=torch.uint8, device="cuda"), torch.ones(2, 1, device="cuda"),
                    _i32([[0, 1]]))
    with pytest.raises(api.CSAError) as e:           # blocks of 24 rows
        api.csa_cache_write(h, odd, x[:, :1].contiguous(), cu, p0)
    assert e.value.code == -2
    dim = api.Cache(torch.zeros(2, 1, 16, 96, dtype=torch.uint8, device="cuda"), torch.ones(2, 1, device="cuda"),
                    _i32([[0, 1]]))
    with pytest.raises(api.CSAError) as e:           # 96 dims
        api.csa_cache_read(h, dim, cu, p0, torch.zeros(4, 1, 96, device="cuda"))
    assert e.value.code == -2
    api.csa_cache_write(h, cache, x[:0], _i32([0, 0]), p0, x_v=x[:0])   # no rows: nothing to do
    assert h.device_status() == 0
