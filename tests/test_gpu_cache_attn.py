"""csa_cache_attn_fwd against the plain 64-bit model: compressed entries (all, or listed) and
windows, grouped and shared heads, one token to chunks, ragged and odd sizes, masked garbage."""
import math

import numpy as np
import pytest
import torch

from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from compressed_sparse_attention_compress_gb300 import api  # noqa: E402


def _i32(v):
    return torch.from_numpy(np.asarray(v, np.int32)).cuda()


class Call:
    """One call with random caches, and the model's answer to it."""

    def __init__(self, seed, ctx, n, H, H_kv, d, block, shared, fp32=False, ratio=0, topk=0, window=0, sink=False,
                 pad=3, max_blocks=None):
        rng = self.rng = np.random.default_rng(seed)
        self.h = api.Handle(0)
        B = len(ctx)
        self.ctx, self.n, self.ratio, self.window = ctx, n, ratio, window
        self.cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.T = int(self.cu[-1]) + pad
        rows = [c + m for c, m in zip(ctx, n)]
        self.scmp = ch.Setup(seed + 1, B, [r // ratio for r in rows], H_kv, d, block, shared) if ratio else None
        self.sraw = ch.Setup(seed + 2, B, rows, H_kv, d, block, shared, max_blocks) if window else None
        self.cmp = api.Cache(**self.scmp.tensors()) if ratio else None
        self.raw = api.Cache(**self.sraw.tensors()) if window else None
        q = rng.standard_normal((self.T, H, d))
        self.q = torch.from_numpy(q.astype(np.float32)).cuda()
        self.q = self.q if fp32 else self.q.to(torch.bfloat16)
        self.sink = torch.from_numpy(rng.standard_normal(H).astype(np.float32)).cuda() if sink else None
        self.scale = 1.0 / math.sqrt(d)
        self.idx = None
        if topk:
            idx = np.full((self.T, topk), -1, np.int32)
            for b in range(B):
                for i in range(n[b]):
                    vis = (ctx[b] + i + 1) // ratio
                    m = min(vis, int(rng.integers(0, topk + 1)))
                    idx[self.cu[b] + i, :m] = rng.permutation(vis)[:m]
                    rng.shuffle(idx[self.cu[b] + i])       # -1 anywhere, no order
            self.idx = idx
        self.ws = torch.empty(max(16, api.csa_cache_attn_workspace(self.h, self.T, H, H_kv, d)), dtype=torch.uint8,
                              device="cuda").fill_(0xFF)
        self.out = torch.full_like(self.q, 5.0)
        self.lse = torch.full((self.T, H), 5.0, device="cuda")

    def run(self, base=None, **kw):
        idx = None if self.idx is None else _i32(self.idx if base is None else self.idx + self._base(base))
        args = dict(cmp=self.cmp, raw=self.raw, idx=idx, cu_cmp=None if base is None else _i32(base),
                    ratio=self.ratio, window=self.window, sink=self.sink, lse=self.lse)
        args.update(kw)
        api.csa_cache_attn_fwd(self.h, self.q, _i32(self.cu), _i32(self.ctx), self.scale, self.out, self.ws, **args)

    def _base(self, base):
        add = np.zeros((self.T, 1), np.int32)
        for b in range(len(self.ctx)):
            add[self.cu[b]:self.cu[b + 1]] = base[b]
        return np.where(self.idx >= 0, add, 0)

    def ref(self):
        return ch.attend(self.q.double().cpu().numpy(), self.cu, self.ctx, self.scale,
                         cmp=self.scmp.models() if self.ratio else None, raw=self.sraw.models() if self.window else None,
                         idx=self.idx, ratio=self.ratio, window=self.window,
                         sink=None if self.sink is None else self.sink.double().cpu().numpy())

    def check(self):
        torch.cuda.synchronize()
        assert self.h.device_status() == 0
        ch.check(self.out, self.lse, self.ref(), self.q.dtype)
        end = int(self.cu[-1])
        assert not self.out[end:].any() and torch.isneginf(self.lse[end:]).all()


FULL = 1 << 20
CASES = {
    "one_key": dict(ctx=[0], n=[1], H=1, H_kv=1, d=64, block=16, shared=False, window=1),
    "one_token_each": dict(ctx=[0, 1, 14, 15, 16, 63, 64, 65, 300], n=[1] * 9, H=8, H_kv=2, d=64, block=16,
                           shared=False, window=FULL),
    "grouped_128": dict(ctx=[700, 0, 129], n=[1, 1, 1], H=16, H_kv=2, d=128, block=64, shared=False, window=FULL,
                        sink=True),
    "grouped_5": dict(ctx=[333, 90], n=[1, 2], H=15, H_kv=3, d=128, block=32, shared=False, window=FULL),
    "one_head_each": dict(ctx=[200, 31], n=[3, 1], H=3, H_kv=3, d=64, block=128, shared=False, window=FULL),
    "shared_64": dict(ctx=[511, 40], n=[1, 1], H=64, H_kv=1, d=128, block=64, shared=True, window=FULL),
    "shared_128": dict(ctx=[100], n=[2], H=128, H_kv=1, d=64, block=16, shared=True, window=FULL, sink=True),
    "heads_33": dict(ctx=[77], n=[1], H=33, H_kv=1, d=128, block=16, shared=False, window=FULL),
    "window_77": dict(ctx=[0, 76, 77, 500, 1023], n=[1, 2, 3, 1, 4], H=4, H_kv=1, d=128, block=64, shared=True,
                      window=77, sink=True),
    "window_1": dict(ctx=[9, 130], n=[2, 1], H=4, H_kv=4, d=64, block=16, shared=False, window=1),
    "fp32": dict(ctx=[0, 255, 70], n=[1, 5, 2], H=8, H_kv=4, d=64, block=16, shared=False, window=64, fp32=True,
                 sink=True),
    "fp32_128": dict(ctx=[300], n=[2], H=64, H_kv=1, d=128, block=64, shared=True, window=128, ratio=4, fp32=True),
    "hca": dict(ctx=[126, 127, 1000, 0], n=[1, 1, 1, 1], H=64, H_kv=1, d=128, block=32, shared=True, ratio=128,
                window=128, sink=True),
    "dense_ratio_4": dict(ctx=[1999, 2, 257], n=[1, 1, 3], H=64, H_kv=1, d=128, block=64, shared=True, ratio=4,
                          window=128),
    "entries_only": dict(ctx=[5, 0, 400], n=[1, 2, 3], H=8, H_kv=2, d=64, block=16, shared=False, ratio=4),
    "causal_by_entries": dict(ctx=[0, 83], n=[40, 7], H=4, H_kv=2, d=128, block=32, shared=False, ratio=1),
    "csa": dict(ctx=[2000, 3, 0, 700], n=[1, 1, 1, 2], H=64, H_kv=1, d=128, block=64, shared=True, ratio=4, topk=100,
                window=128, sink=True),
    "csa_entries_only": dict(ctx=[800, 2, 90], n=[2, 1, 1], H=16, H_kv=1, d=64, block=16, shared=False, ratio=4,
                             topk=65),
    "csa_fp32": dict(ctx=[500], n=[3], H=4, H_kv=1, d=64, block=16, shared=False, ratio=4, topk=33, window=64,
                     fp32=True),
    "csa_grouped": dict(ctx=[640, 30], n=[2, 1], H=12, H_kv=4, d=128, block=32, shared=False, ratio=4, topk=48,
                        window=16),
    "chunk": dict(ctx=[0, 37, 190], n=[130, 65, 1], H=8, H_kv=2, d=128, block=64, shared=False, window=FULL),
    "chunk_window": dict(ctx=[100, 0], n=[97, 33], H=16, H_kv=2, d=64, block=16, shared=False, window=40, sink=True),
    "chunk_shared_64": dict(ctx=[50], n=[70], H=64, H_kv=1, d=128, block=64, shared=True, ratio=4, window=32),
    "chunk_odd_group": dict(ctx=[3], n=[50], H=21, H_kv=3, d=64, block=32, shared=False, window=FULL, fp32=True),
    "empty_sequences": dict(ctx=[10, 20, 30, 40], n=[0, 2, 0, 0], H=4, H_kv=1, d=64, block=16, shared=True, window=8),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_the_definition(name):
    c = Call(7, **CASES[name])
    c.run()
    c.check()


def test_global_rows_as_the_top_k_writes_them():
    c = Call(11, ctx=[800, 300], n=[2, 1], H=64, H_kv=1, d=128, block=64, shared=True, ratio=4, topk=70, window=64)
    c.run(base=[40, 1000, 1100])
    c.check()


def test_garbage_in_masked_places_does_not_reach_the_output():
    # NaN codes in every row that no query sees: behind the last row, before the window, in entries not
    # listed or not yet visible, in blocks of other sequences; and in V rows that a later query of the chunk sees
    for kw in (dict(ctx=[200, 45], n=[1, 3], H=8, H_kv=1, d=64, block=16, shared=False, window=30),
               dict(ctx=[200, 45], n=[2, 1], H=64, H_kv=1, d=128, block=64, shared=True, ratio=4, window=30),
               dict(ctx=[900, 45], n=[1, 2], H=16, H_kv=1, d=128, block=64, shared=True, ratio=4, topk=40, window=20)):
        c = Call(13, **kw)
        for s, cache, is_cmp in ((c.scmp, c.cmp, True), (c.sraw, c.raw, False)):
            if s is None:
                continue
            seen = np.zeros((s.n, s.block), bool)
            for b in range(len(c.ctx)):
                for i in range(c.n[b]):
                    p = c.ctx[b] + i
                    if is_cmp:
                        e = np.arange((p + 1) // c.ratio)
                        if c.idx is not None:
                            e = c.idx[c.cu[b] + i]
                            e = e[e >= 0]
                    else:
                        e = np.arange(max(0, p - c.window + 1), p + 1)
                    seen[s.table[b][e // s.block], e % s.block] = True
            for t in (cache.k, cache.v):
                if t is not None:
                    t.copy_(torch.where(torch.from_numpy(seen).cuda()[:, None, :, None], t, torch.full_like(t, 0x7F)))
        c.run()
        c.check()


@pytest.mark.parametrize("d,H,H_kv,shared", [(128, 8, 1, False), (64, 4, 2, False), (128, 64, 1, True)])
def test_nan_rows_reach_the_queries_that_see_them_and_no_others(d, H, H_kv, shared):
    c = Call(17, ctx=[20], n=[40], H=H, H_kv=H_kv, d=d, block=16, shared=shared, window=FULL)
    blk, r = c.sraw.table[0][41 // 16], 41 % 16
    for kind, (code, _) in enumerate(c.sraw.kinds):
        code[blk, :, r, 5] = 0x7F if kind == 0 or H_kv == 1 else code[blk, :, r, 5]
    c.raw = api.Cache(**c.sraw.tensors())
    c.run()
    torch.cuda.synchronize()
    out = c.out.float().cpu().numpy()
    assert np.isfinite(out[:21]).all()                       # positions 20..40 come before the row
    assert np.isnan(out[21:40]).any(axis=(1, 2)).all()
    ref = c.ref()
    good = tuple(x[:21] for x in ref)
    ch.check(c.out[:21], c.lse[:21], good, c.q.dtype)


def test_scales_far_apart_and_scores_far_apart():
    # a block whose V scale is 2^80 times another's, and scores that climb by hundreds from block to block
    for fp32 in (False, True):
        c = Call(19, ctx=[159], n=[1], H=8, H_kv=2, d=64, block=16, shared=False, window=FULL, fp32=fp32)
        for b, e in enumerate([0, -80, 40, 0, 0, -40, 10, 60, 0, -100]):
            c.sraw.kinds[1][1][c.sraw.table[0][b]] *= 2.0 ** e
        for b in range(10):
            c.sraw.kinds[0][1][c.sraw.table[0][b]] = 2.0 ** (b - 13)
        c.raw = api.Cache(**c.sraw.tensors())
        c.run()
        c.check()


def test_an_entry_listed_twice_counts_twice_and_bad_entries_are_skipped():
    c = Call(23, ctx=[400], n=[1], H=16, H_kv=1, d=64, block=16, shared=True, ratio=4, topk=40, window=8, pad=0)
    c.idx[0, :] = -1
    c.idx[0, :6] = [3, 3, 99, 3, 7, 99]
    c.run()
    c.check()
    c.idx[0, 10:13] = [100, 5000, 2 ** 31 - 1]               # entry 100 is not complete at position 400
    c.run()
    assert c.h.device_status() == -6
    c.h.device_status()
    ref = c.ref()                                            # the model leaves them out
    ch.check(c.out, c.lse, ref, c.q.dtype)


def test_bad_positions_blocks_and_lists_raise_the_status():
    c = Call(29, ctx=[10, 20, 30], n=[1, 1, 1], H=4, H_kv=1, d=64, block=16, shared=True, window=64, pad=0)
    bad = [-1, 20, 64]
    api.csa_cache_attn_fwd(c.h, c.q, _i32(c.cu), _i32(bad), c.scale, c.out, c.ws, raw=c.raw, window=64, lse=c.lse)
    assert c.h.device_status() == -6
    ref = c.ref()
    assert not c.out[0].any() and not c.out[2].any() and torch.isneginf(c.lse[0]).all()
    ch.check(c.out[1:2], c.lse[1:2], tuple(x[1:2] for x in ref), c.q.dtype)
    c.sraw.t_table[1, 0] = c.sraw.n + 5                      # the first 16 rows of sequence 1 are lost
    c.run()
    assert c.h.device_status() == -6
    m = c.sraw.models()
    K = m[0].rows(1, np.arange(16, 21))[:, 0]
    x = c.q[1].double().cpu().numpy() @ K.T * c.scale
    w = np.exp(x - x.max(1, keepdims=True))
    np.testing.assert_allclose(c.out[1].float().cpu().numpy(), w @ K / w.sum(1, keepdims=True), atol=0.03)


def test_run_to_run_streams_graphs_and_two_workspaces():
    kw = dict(ctx=[3000, 1700, 20], n=[1, 1, 1], H=32, H_kv=4, d=128, block=64, shared=False, window=FULL)
    c, e = Call(31, **kw), Call(31, **kw)
    c.run()
    torch.cuda.synchronize()
    first, z = c.out.clone(), c.lse.clone()
    for _ in range(3):
        c.run()
    torch.cuda.synchronize()
    assert torch.equal(first, c.out) and torch.equal(z, c.lse)
    streams = [torch.cuda.Stream() for _ in range(2)]        # two calls at once, a workspace each
    for _ in range(5):
        for x, st in zip((c, e), streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                x.run()
    torch.cuda.synchronize()
    assert torch.equal(first, c.out) and torch.equal(first, e.out)
    cu, p0 = _i32(c.cu), _i32(c.ctx)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        api.csa_cache_attn_fwd(c.h, c.q, cu, p0, c.scale, c.out, c.ws, raw=c.raw, window=FULL, lse=c.lse)
    c.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, c.out)
    p0.copy_(_i32([100, 1699, 0]))                           # replayed with other lengths
    g.replay()
    torch.cuda.synchronize()
    c.ctx = [100, 1699, 0]
    c.check()


def test_without_lse_and_refusals():
    c = Call(37, ctx=[100], n=[1], H=8, H_kv=2, d=64, block=16, shared=False, window=50)
    c.run(lse=None)
    torch.cuda.synchronize()
    ch.check(c.out, None, c.ref(), c.q.dtype)
    with pytest.raises(ValueError):
        c.run(raw=None)
    with pytest.raises(api.CSAError):
        c.run(window=0)
    with pytest.raises(ValueError):
        c.run(sink=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        c.run(lse=torch.zeros(c.T, 8))
    q = c.q
    c.q = q.half()
    with pytest.raises(TypeError):
        c.run()
    c.q = torch.zeros(c.T, 8, 128, device="cuda")[..., ::2]
    with pytest.raises(ValueError):
        c.run()


def test_long_caches_past_31_bits_of_codes():
    # 2^31 codes and more in one cache: the offsets take 64 bits
    n, H_kv, block, d = 140000, 2, 64, 128
    k = torch.zeros(n, H_kv, block, d, dtype=torch.uint8, device="cuda")
    ks = torch.full((n, H_kv), 2.0 ** -8, device="cuda")
    table = torch.tensor([[n - 1, 5, n - 2]], dtype=torch.int32, device="cuda")
    c = api.Cache(k, ks, table)
    h = api.Handle(0)
    x = torch.randn(150, H_kv, d, device="cuda").to(torch.bfloat16)
    cu, p0 = _i32([0, 150]), _i32([0])
    api.csa_cache_write(h, c, x, cu, p0)
    back = torch.empty_like(x)
    api.csa_cache_read(h, c, cu, p0, back)
    err = (back.float() - x.float()).abs().max().item()
    assert err <= 2.0 ** -4 * x.abs().max().item()
    q = torch.randn(1, 4, d, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    ws = torch.empty(max(16, api.csa_cache_attn_workspace(h, 1, 4, H_kv, d)), dtype=torch.uint8, device="cuda")
    api.csa_cache_attn_fwd(h, q, _i32([0, 1]), _i32([149]), d ** -0.5, out, ws, raw=c, window=FULL)
    assert h.device_status() == 0
    K = back.double().repeat_interleave(2, 1)
    w = torch.softmax(torch.einsum("hd,khd->hk", q[0].double(), K) * d ** -0.5, -1)
    ref = torch.einsum("hk,khd->hd", w, K)
    assert (out[0].double() - ref).abs().max().item() <= 2.0 ** -7 * ref.abs().max().item()
