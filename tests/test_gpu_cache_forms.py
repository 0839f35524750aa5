"""The forms of csa_cache_attn_fwd (16, 32, 64 and 128 rows of an item; K = V or not) and of
csa_cache_write (few or many rows a sequence) where each can go wrong: far scales, NaN, rows of other
magnitudes, many sequences, items cut among CTAs."""
import numpy as np
import pytest
import torch

from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from compressed_sparse_attention_compress_gb300 import api  # noqa: E402
from tests.test_gpu_cache_attn import FULL, Call, _i32  # noqa: E402

# rows of an item = heads of a group x queries a sequence on average (the capacity rows count)
FORMS = {
    "16": dict(ctx=[300, 129], n=[1, 1], H=8, H_kv=1, shared=False),
    "16_shared": dict(ctx=[300, 129], n=[1, 1], H=16, H_kv=1, shared=True),
    "32": dict(ctx=[300, 129], n=[4, 4], H=8, H_kv=1, shared=False),
    "64": dict(ctx=[300, 129], n=[8, 8], H=16, H_kv=2, shared=False),
    "64_shared": dict(ctx=[300, 129], n=[1, 1], H=64, H_kv=1, shared=True),
    "64_one_group_of_33": dict(ctx=[300, 129], n=[1, 1], H=33, H_kv=1, shared=False),
    "128": dict(ctx=[300, 129], n=[21, 20], H=16, H_kv=2, shared=False),
    "128_shared": dict(ctx=[300, 129], n=[1, 2], H=128, H_kv=1, shared=True),
    "128_one_head": dict(ctx=[300, 2], n=[140, 131], H=1, H_kv=1, shared=False),
    "128_odd_group": dict(ctx=[77, 0], n=[30, 29], H=15, H_kv=3, shared=False),
    "256": dict(ctx=[40], n=[70], H=64, H_kv=16, shared=True),
}


def call(form, seed, **kw):
    return Call(seed, **{**dict(d=128, block=32, window=FULL, pad=0), **FORMS[form], **kw})


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("kind", ["all", "window", "entries_and_window", "listed"])
def test_against_the_definition(form, kind):
    kw = dict(all=dict(), window=dict(window=45, sink=True), entries_and_window=dict(ratio=4, window=20, sink=True),
              listed=dict(ratio=2, topk=50, window=33))[kind]
    c = call(form, 3, **kw)
    c.run()
    c.check()


@pytest.mark.parametrize("form", list(FORMS))
def test_scales_and_scores_far_apart(form):
    c = call(form, 5, ratio=4, window=60)
    for s in (c.scmp, c.sraw):
        for b in range(len(c.ctx)):
            for j, blk in enumerate(s.table[b]):
                if blk >= 0:
                    s.kinds[-1][1][blk] *= 2.0 ** [0, -80, 40, 0, -40, 10, 60, -100, 3][j % 9]
                    if not c.sraw.shared:
                        s.kinds[0][1][blk] *= 2.0 ** (j - 6)
    if c.sraw.shared:  # the scores carry the scales too: keep them within float32's range
        c.scale *= 2.0 ** -30
    c.cmp, c.raw = api.Cache(**c.scmp.tensors()), api.Cache(**c.sraw.tensors())
    c.run()
    c.check()


@pytest.mark.parametrize("form", list(FORMS))
def test_nan_rows_reach_the_rows_that_see_them_and_no_others(form):
    c = call(form, 7)
    b = len(c.ctx) - 1
    at = c.ctx[b] + c.n[b] // 2                              # a row that the first half of the queries does not see
    blk, r = c.sraw.table[b][at // 32], at % 32
    c.sraw.kinds[-1][0][blk, 0, r, 37] = 0xFF                # of V (of K = V): KV head 0 alone
    c.raw = api.Cache(**c.sraw.tensors())
    c.run()
    torch.cuda.synchronize()
    bad = torch.isnan(c.out.float()).cpu().numpy()           # [T, H, d]
    G = c.q.shape[1] // c.sraw.kinds[0][0].shape[1]
    want = np.zeros_like(bad)
    first = c.cu[b] + at - c.ctx[b]
    # K = V: the score is NaN, hence the row; else dim 37 alone
    want[first:c.cu[b + 1], :G, slice(None) if c.sraw.shared else 37] = True
    assert np.array_equal(bad, want)
    ref = c.ref()
    sel = ~want.any(axis=2)
    for i in range(c.T):
        hs = np.flatnonzero(sel[i])
        if len(hs):
            ch.check(c.out[i][hs], c.lse[i][hs], tuple(x[i][hs] for x in ref), c.q.dtype)


@pytest.mark.parametrize("form", list(FORMS))
def test_queries_that_are_not_finite_or_of_other_sizes(form):
    c = call(form, 9, ratio=4, window=30)
    T, H = c.q.shape[:2]
    size = torch.from_numpy(2.0 ** np.random.default_rng(1).integers(-12, 7, (T, H, 1))).cuda().to(c.q.dtype)
    c.q.mul_(size)                                           # exact: powers of two
    good = c.q.clone()
    t = T // 2
    c.q[t, H // 2, 5] = float("nan")
    c.q[0, 0, 0] = float("inf")
    c.run()
    torch.cuda.synchronize()
    bad = torch.zeros(T, H, dtype=torch.bool, device="cuda")
    bad[t, H // 2] = bad[0, 0] = True
    assert torch.equal(torch.isnan(c.out.float()).all(-1), bad) and torch.equal(torch.isnan(c.out.float()).any(-1), bad)
    c.q = good
    ref = c.ref()
    keep = ~bad.cpu().numpy()
    for i in range(T):
        hs = np.flatnonzero(keep[i])
        if len(hs):
            ch.check(c.out[i][hs], c.lse[i][hs], tuple(x[i][hs] for x in ref), c.q.dtype)


@pytest.mark.parametrize("form", ["16", "64_shared", "128"])
def test_two_graphs_share_a_workspace_and_replay_with_other_lengths(form):
    c, e = call(form, 11, max_blocks=24), call(form, 12, max_blocks=24)
    e.ws = c.ws
    cu, p0 = _i32(c.cu), [_i32(c.ctx), _i32(e.ctx)]
    torch.cuda.synchronize()
    graphs = []
    for x, p in zip((c, e), p0):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(2):
                api.csa_cache_attn_fwd(x.h, x.q, cu, p, x.scale, x.out, x.ws, raw=x.raw, window=FULL, lse=x.lse)
        graphs.append(g)
    for ctx in (c.ctx, [7] * len(c.ctx), [0] * len(c.ctx), c.ctx):
        for g, x, p in zip(graphs, (c, e), p0):
            p.copy_(_i32(ctx))
            x.out.fill_(9.0)
            g.replay()
        for x in (c, e):
            x.ctx = ctx
            x.check()


@pytest.mark.parametrize("H,H_kv,shared,n", [(4, 2, False, 1), (64, 1, True, 1), (8, 1, False, 9)])
def test_many_ragged_sequences(H, H_kv, shared, n):
    rng = np.random.default_rng(2)
    B = 301
    c = Call(13, ctx=[int(x) for x in rng.integers(0, 150, B)], n=[int(x) for x in rng.integers(0, n + 1, B)], H=H,
             H_kv=H_kv, d=128, block=16, shared=shared, window=FULL, pad=7)
    c.run()
    c.check()


@pytest.mark.parametrize("H,d,fp32", [(2, 64, True), (4, 128, False), (17, 128, False)])
def test_more_sequences_than_shared_memory_holds(H, d, fp32):
    # items of one tile, which no CTA cuts: the same bits as in calls of 2000 sequences
    B, block, n = 26000, 16, 64
    g = torch.Generator().manual_seed(4)
    k = torch.randint(0, 0x7E, (n, 1, block, d), generator=g, dtype=torch.uint8).cuda()
    ks = torch.full((n, 1), 2.0 ** -7, device="cuda")
    table = torch.randint(0, n, (B, 4), generator=g, dtype=torch.int32).cuda()
    ctx = torch.randint(0, 60, (B,), generator=g, dtype=torch.int32).cuda()
    dt = torch.float32 if fp32 else torch.bfloat16
    q = torch.randn(B + 5, H, d, generator=g).cuda().to(dt)
    h = api.Handle(0)

    def run(lo, hi, rows):
        out = torch.full_like(rows, 3.0)
        ws = torch.empty(api.csa_cache_attn_workspace(h, len(rows), H, 1, d), dtype=torch.uint8, device="cuda")
        api.csa_cache_attn_fwd(h, rows, _i32(np.arange(hi - lo + 1)), ctx[lo:hi].clone(), d ** -0.5, out, ws,
                               raw=api.Cache(k, ks, table[lo:hi].clone()), window=FULL)
        return out

    whole = run(0, B, q)
    for lo in range(0, B, 2000):
        assert torch.equal(whole[lo:lo + 2000], run(lo, lo + 2000, q[lo:lo + 2000].clone()))
    assert not whole[B:].any() and h.device_status() == 0


def test_no_sequences():
    c = call("64_shared", 1, pad=6)
    none = _i32([0])
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    x = c.q[:, :1].contiguous()
    before = c.raw.k.clone()
    api.csa_cache_write(c.h, c.raw, x, none, empty)
    api.csa_cache_read(c.h, c.raw, none, empty, x)
    api.csa_cache_attn_fwd(c.h, c.q, none, empty, c.scale, c.out, c.ws, raw=c.raw, window=FULL, lse=c.lse)
    assert c.h.device_status() == 0
    assert torch.equal(before, c.raw.k) and not x.any() and not c.out.any() and torch.isneginf(c.lse).all()
    nothing = c.q[:0].contiguous()
    c.out.fill_(2.0)
    api.csa_cache_attn_fwd(c.h, nothing, none, empty, c.scale, nothing, None, raw=c.raw, window=FULL)
    assert c.h.device_status() == 0 and (c.out == 2.0).all()


def test_items_cut_among_ctas_and_whole_ones_agree():
    # the same query and cache alone (cut into pieces) and among many (whole): the same values up to the joins
    for H, H_kv, shared in ((8, 1, False), (64, 1, True)):
        kw = dict(H=H, H_kv=H_kv, d=128, block=64, shared=shared, window=FULL)
        c = Call(17, ctx=[9000], n=[1], pad=0, **kw)
        c.run()
        c.check()
        e = Call(17, ctx=[9000], n=[1], pad=0, **kw)
        B = 400
        e.q, e.out, e.lse = c.q.repeat(B, 1, 1), c.out.repeat(B, 1, 1).zero_(), c.lse.repeat(B, 1).zero_()
        e.raw = api.Cache(e.raw.k, e.raw.k_scale, e.raw.table.repeat(B, 1), v=e.raw.v, v_scale=e.raw.v_scale)
        ws = torch.empty(api.csa_cache_attn_workspace(e.h, B, H, H_kv, 128), dtype=torch.uint8, device="cuda")
        api.csa_cache_attn_fwd(e.h, e.q, _i32(np.arange(B + 1)), _i32([9000] * B), e.scale, e.out, ws, raw=e.raw,
                               window=FULL, lse=e.lse)
        torch.cuda.synchronize()
        assert e.h.device_status() == 0
        ref = c.ref()
        for b in (0, 1, 151, 152, 399):
            ch.check(e.out[b:b + 1], e.lse[b:b + 1], ref, e.q.dtype)


@pytest.mark.parametrize("n", [1, 15, 16, 17, 64, 200])
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_writes_of_few_and_of_many_rows(n, fp32, shared):
    rng = np.random.default_rng(n)
    B, H_kv, d, block = 5, 3, 64, 32
    ctx = [0, 31, 32, 45, 64]
    s = ch.Setup(1, B, [p + n for p in ctx], H_kv, d, block, shared)
    cache, models = api.Cache(**s.tensors()), s.models()
    x = rng.standard_normal((2, B * n, H_kv, d)) * np.exp(3 * rng.standard_normal((2, B * n, H_kv, 1)))
    x = torch.from_numpy(x.astype(np.float32))
    x[0, 0, 0, 0], x[0, n - 1, 1, 5], x[1, 0, 2, 63] = float("inf"), float("nan"), float("-inf")
    x[0, n:2 * n, 0] = 0.0                                    # a head whose rows are all zero
    x = x if fp32 else x.to(torch.bfloat16)
    cu = np.arange(B + 1) * n
    h = api.Handle(0)
    api.csa_cache_write(h, cache, x[0].cuda(), _i32(cu), _i32(ctx), x_v=None if shared else x[1].cuda())
    assert h.device_status() == 0
    for kind, (codes, scale) in enumerate([(cache.k, cache.k_scale), (cache.v, cache.v_scale)][:1 if shared else 2]):
        models[kind].write(x[kind].double().numpy(), cu, ctx)
        got, sc = codes.cpu().numpy(), scale.double().cpu().numpy()
        for b in range(B):
            p = np.arange(ctx[b] + n)
            blk = s.table[b][p // block]
            assert np.array_equal(sc[blk], models[kind].scale[blk])
            g, w = got[blk, :, p % block], models[kind].codes[blk, :, p % block]
            nan = (w & 0x7F) == 0x7F
            assert np.array_equal((g & 0x7F) == 0x7F, nan) and np.array_equal(g[~nan], w[~nan])
