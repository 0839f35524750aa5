"""The serving calls as a program makes them: a prompt is compressed and its entries and raw rows go into
the caches, then tokens are decoded one at a time -- select, write, attend -- beside the existing calls."""
import math

import numpy as np
import pytest
import torch

from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from compressed_sparse_attention_compress_gb300 import api  # noqa: E402

RATIO, TOPK, WINDOW, H, D, H_I, D_I, BLOCK = 4, 16, 32, 64, 128, 8, 64, 32


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


class Layer:
    """Rows of a few sequences, drawn once; the packed rows up to given lengths."""

    def __init__(self, lengths, extra):
        g = torch.Generator().manual_seed(3)
        draw = lambda *s: torch.randn(*s, generator=g).to("cuda", torch.bfloat16)
        n = [x + extra for x in lengths]
        self.x, self.z = [draw(m, D) for m in n], [draw(m, D) for m in n]
        self.xi, self.zi = [draw(m, D_I) for m in n], [draw(m, D_I) for m in n]
        self.q, self.qi, self.w = ([draw(m, *s) for m in n] for s in ((H, D), (H_I, D_I), (H_I,)))
        self.bias = torch.randn(2 * RATIO, D, generator=g).cuda()
        self.bias_i = torch.randn(2 * RATIO, D_I, generator=g).cuda()
        self.sink = torch.randn(H, generator=g).cuda()
        B, most = len(lengths), max(n)
        self.raw = self._cache(g, B, most)
        self.cmp = self._cache(g, B, most // RATIO)

    @staticmethod
    def _cache(g, B, rows):
        width = -(-rows // BLOCK)
        table = torch.randperm(B * width, generator=g).to(torch.int32).view(B, width).cuda()
        k = torch.randint(0, 256, (B * width, 1, BLOCK, D), generator=g, dtype=torch.uint8).cuda()  # what was there
        return api.Cache(k, torch.full((B * width, 1), 7.0, device="cuda"), table)

    def packed(self, rows, lengths, first=None):
        return torch.cat([r[(first[b] if first else 0):lengths[b]] for b, r in enumerate(rows)])

    def entries(self, h, lengths):
        cu = _i32(np.concatenate([[0], np.cumsum(lengths)]))
        cap = sum(lengths) // RATIO + 2
        cu_cmp = torch.zeros(len(lengths) + 1, dtype=torch.int32, device="cuda")
        kv = torch.zeros(cap, D, dtype=torch.bfloat16, device="cuda")
        ki = torch.zeros(cap, D_I, dtype=torch.bfloat16, device="cuda")
        p = lambda r: self.packed(r, lengths)
        api.csa_compress_pair(h, p(self.x), p(self.z), self.bias, p(self.xi), p(self.zi), self.bias_i, cu, max(lengths),
                              RATIO, True, cu_cmp, kv, ki)
        return cu, cu_cmp, kv, ki

    def models(self, cache):
        m = ch.Model(cache.k.cpu().numpy(), cache.k_scale.cpu().numpy(), cache.table.cpu().numpy())
        return m, m


def test_prompt_then_tokens():
    lengths, steps = [150, 37, 3], 6
    L = Layer(lengths, steps)
    h, hs = api.Handle(0), api.Handle(0)
    B, scale = len(lengths), 1.0 / math.sqrt(D)
    zero = _i32([0] * B)

    # the prompt: all entries, all rows, every query
    cu, cu_cmp, kv, ki = L.entries(h, lengths)
    T = sum(lengths)
    api.csa_cache_write(h, L.cmp, kv[:, None], cu_cmp, zero)
    raw = L.packed(L.x, lengths)
    api.csa_cache_write(h, L.raw, raw[:, None], cu, zero)
    idx = torch.empty(T, TOPK, dtype=torch.int32, device="cuda")
    api.csa_indexer_topk(h, L.packed(L.qi, lengths), L.packed(L.w, lengths), ki, cu, cu_cmp, max(lengths), RATIO, TOPK, idx)
    q = L.packed(L.q, lengths)
    ws = torch.empty(api.csa_cache_attn_workspace(h, T, H, 1, D), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(T, H, device="cuda")
    api.csa_cache_attn_fwd(h, q, cu, zero, scale, out, ws, cmp=L.cmp, raw=L.raw, idx=idx, cu_cmp=cu_cmp, ratio=RATIO,
                           window=WINDOW, sink=L.sink, lse=lse)
    assert h.device_status() == 0
    n_cmp = cu_cmp.cpu().numpy()
    ref = ch.attend(q.double().cpu().numpy(), cu.cpu().numpy(), [0] * B, scale, cmp=L.models(L.cmp),
                    raw=L.models(L.raw), idx=idx.cpu().numpy(), base=n_cmp, ratio=RATIO, window=WINDOW,
                    sink=L.sink.double().cpu().numpy())
    ch.check(out, lse, ref, q.dtype)

    # the training call on the rows as the caches hold them (their values are exact in bf16)
    back_cmp, back_raw = torch.zeros_like(kv)[:, None], torch.empty_like(raw)[:, None]
    api.csa_cache_read(h, L.cmp, cu_cmp, zero, back_cmp)
    api.csa_cache_read(h, L.raw, cu, zero, back_raw)
    out2, lse2 = torch.empty_like(q), torch.empty(T, H, device="cuda")
    api.csa_sparse_attn_fwd(h, q, back_cmp[:, 0], back_raw[:, 0], idx, cu, cu_cmp, max(lengths), RATIO, WINDOW, scale, out2,
                            lse2, sink=L.sink)
    # both outputs are rounded to bf16 (2^-8 each); its weights have 8 bits (2^-8), this call's 11 (2^-11)
    bound = 2 * 2.0 ** -8 * np.abs(ref[0]) + (2.0 ** -8 + 2.0 ** -11 + 8 * ref[3][..., None]) * ref[2] * 1.01 + ref[4]
    assert (np.abs(out.double().cpu().numpy() - out2.double().cpu().numpy()) <= bound).all()

    # tokens: one query a sequence; entries are added as they become complete
    one = _i32(np.arange(B + 1))
    for step in range(steps):
        pos = [n + step for n in lengths]
        now = [p + 1 for p in pos]
        p0 = _i32(pos)
        api.csa_cache_write(h, L.raw, L.packed(L.x, now, pos)[:, None], one, p0)
        _, cu_cmp, kv, ki = L.entries(h, now)
        new = [int((p + 1) % RATIO == 0) for p in pos]
        if any(new):
            c = cu_cmp.cpu().numpy()
            rows = torch.cat([kv[c[b + 1] - new[b]:c[b + 1]] for b in range(B)])[:, None]
            api.csa_cache_write(h, L.cmp, rows.contiguous(), _i32(np.concatenate([[0], np.cumsum(new)])),
                                _i32([p // RATIO for p in pos]))
        idx = torch.empty(B, TOPK, dtype=torch.int32, device="cuda")
        hs.set_position_offsets(p0, int(cu_cmp[-1]))
        api.csa_indexer_topk(hs, L.packed(L.qi, now, pos), L.packed(L.w, now, pos), ki, one, cu_cmp, max(now), RATIO, TOPK,
                             idx)
        q = L.packed(L.q, now, pos)
        out, lse = torch.empty_like(q), torch.empty(B, H, device="cuda")
        api.csa_cache_attn_fwd(h, q, one, p0, scale, out, ws, cmp=L.cmp, raw=L.raw, idx=idx, cu_cmp=cu_cmp, ratio=RATIO,
                               window=WINDOW, sink=L.sink, lse=lse)
        assert h.device_status() == 0 and hs.device_status() == 0
        for b in range(B):  # what the selection lists is what the attention reads
            got = idx[b].cpu().numpy()
            assert (got >= 0).sum() == min(TOPK, now[b] // RATIO)
        ref = ch.attend(q.double().cpu().numpy(), np.arange(B + 1), pos, scale, cmp=L.models(L.cmp), raw=L.models(L.raw),
                        idx=idx.cpu().numpy(), base=cu_cmp.cpu().numpy(), ratio=RATIO, window=WINDOW,
                        sink=L.sink.double().cpu().numpy())
        ch.check(out, lse, ref, q.dtype)


def test_step_on_another_stream_in_a_graph():
    # two layers that share a workspace, written and attended to on a side stream, captured once and replayed
    B, H_kv, Hq, d, ctx = 3, 2, 8, 128, 70
    h = api.Handle(0)
    setups = [ch.Setup(5 + i, B, [ctx + 8] * B, H_kv, d, 64, False) for i in range(2)]
    caches = [api.Cache(**s.tensors()) for s in setups]
    models = [s.models() for s in setups]
    g = torch.Generator().manual_seed(1)
    x = [torch.zeros(2, B, H_kv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q = [torch.zeros(B, Hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    out = [torch.zeros_like(q[0]) for _ in range(2)]
    cu, p0 = _i32(np.arange(B + 1)), _i32([ctx, 5, 0])
    ws = torch.empty(api.csa_cache_attn_workspace(h, B, Hq, H_kv, d), dtype=torch.uint8, device="cuda")

    def step():
        for i in range(2):
            api.csa_cache_write(h, caches[i], x[i][0], cu, p0, x_v=x[i][1])
            api.csa_cache_attn_fwd(h, q[i], cu, p0, 0.1, out[i], ws, raw=caches[i], window=64)
        p0.add_(1)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    pos = np.array([ctx, 5, 0])
    for _ in range(6):
        for i in range(2):
            x[i].copy_(torch.randn(x[i].shape, generator=g).to(torch.bfloat16) * 2.0)
            q[i].copy_(torch.randn(q[i].shape, generator=g).to(torch.bfloat16))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        assert h.device_status() == 0
        for i in range(2):
            for kind in range(2):
                models[i][kind].write(x[i][kind].double().cpu().numpy(), np.arange(B + 1), pos)
            ref = ch.attend(q[i].double().cpu().numpy(), np.arange(B + 1), pos, 0.1, raw=models[i], window=64)
            ch.check(out[i], None, ref, torch.bfloat16)
        pos = pos + 1
