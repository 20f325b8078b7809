"""tq_chunk_attention against plain attention in 64 bits over the oracle's decompression of
the same cache.

Bound: attention64.py's, with the decompressed keys and values off by their own roundings
(u = 2^-11): the rotation's entries and the levels are rounded to fp16, and a row of R has
norm 1, so a coordinate of n/sqrt(d) R c moves by at most 2 u times that vector's norm; the
result is rounded once more (u of itself)."""
import math
import random

import numpy as np
import pytest

from attention64 import U16, attend64, bound, rms_bound
from parity import gpu_compress, gpu_ctx, record

pytestmark = pytest.mark.gpu


def _tq():
    from kv_cache_vector_02_b200 import tq
    return tq


class Case:
    """A cache of ragged sequences written by libtq, its 64-bit decompression, and queries."""

    def __init__(self, orc, nq, ctx, G, Hkv, bits=4, rot=0, km=0, seed=0, loud=1.0, spare=3):
        import torch
        self.nq, self.lens, self.G, self.Hkv = nq, ctx, G, Hkv
        self.c = gpu_ctx(bits, 31, rot, km)
        o = orc.Oracle(128, bits, 31, rot=rot, key_mode=km)
        rng = np.random.default_rng(seed)
        pages = [(n + 15) // 16 for n in ctx]
        nb = sum(pages) + spare
        perm = rng.permutation(nb).astype(np.int32)
        self.max_blocks = max(pages + [1])
        bt = rng.integers(0, nb, (len(ctx), self.max_blocks)).astype(np.int32)  # unused entries: any block
        at = 0
        for b, p in enumerate(pages):
            bt[b, :p] = perm[at:at + p]
            at += p
        self.slots = [(bt[b][np.arange(n) // 16] * 16 + np.arange(n) % 16).astype(np.int32) for b, n in enumerate(ctx)]
        sl = np.concatenate(self.slots + [np.zeros(0, np.int32)])
        g = torch.Generator(device="cuda").manual_seed(seed)
        T = max(len(sl), 1)
        k = (torch.randn((T, Hkv, 128), generator=g, device="cuda") * 1.5).half()
        v = (torch.randn((T, Hkv, 128), generator=g, device="cuda") * 2 + 0.3).half()
        self.k, self.v, self.sl = k[:len(sl)], v[:len(sl)], sl
        self.kc, self.vc = gpu_compress(self.c, k, v, sl if len(sl) else np.full(1, -1, np.int32), nb, Hkv)
        # rows behind a sequence's last token: bytes that decode to NaN norms
        used = np.zeros(nb * 16, bool)
        used[sl] = True
        self._poison(used)
        self.bt = torch.as_tensor(bt, device="cuda")
        self.K, self.V, self.kerr, self.verr = [], [], [], []
        kc, vc = self.kc.cpu().numpy(), self.vc.cpu().numpy()
        kz = kc.copy()
        if km == 0:
            kz[..., -64:] = 0
        for s in self.slots:
            self.K.append(torch.as_tensor(o.decompress_paged(0, kc, s, Hkv), device="cuda"))
            self.V.append(torch.as_tensor(o.decompress_paged(1, vc, s, Hkv), device="cuda"))
            self.kerr.append(2 * U16 * torch.as_tensor(o.decompress_paged(0, kz, s, Hkv), device="cuda").norm(dim=2))
            self.verr.append(2 * U16 * self.V[-1].norm(dim=2))
        self.q = (torch.randn((sum(nq), G * Hkv, 128), generator=g, device="cuda") * loud / math.sqrt(128)).half()
        self.cu = torch.tensor([0] + list(np.cumsum(nq)), dtype=torch.int32, device="cuda")
        self.L = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        self.top = max(ctx + [0])

    def _poison(self, used):
        import torch
        tq = _tq()
        nb = self.kc.shape[0]
        free = torch.as_tensor(~used.reshape(nb, 16), device="cuda")
        for kind, cache in ((0, self.kc), (1, self.vc)):
            n = tq.tq_chunk_bytes(self.c, kind) // 16
            prod = kind == 0 and self.c.key_mode == 0
            code = n - 4 - (20 if prod else 0)
            fields = [code] + ([16] if prod else []) + [4] + ([4] if prod else [])
            at = 0
            for f in fields:
                view = cache[:, :, at:at + 16 * f].view(nb, -1, 16, f)
                view[free[:, None, :, None].expand_as(view)] = 0xFF
                at += 16 * f

    def run(self, fp32=True, out=None, top=None, scale=0.0, ws=None, **kw):
        import torch
        tq = _tq()
        if out is None:
            out = torch.full(self.q.shape, float("nan"), dtype=torch.float32 if fp32 else torch.float16, device="cuda")
        top = self.top if top is None else top
        args = dict(q=self.q, cu_q=self.cu, k_cache=self.kc, v_cache=self.vc, block_table=self.bt, seq_lens=self.L) | kw
        if ws is None:
            ws = torch.full((tq.tq_chunk_workspace_bytes(self.c, args["seq_lens"].shape[0], args["q"].shape[0],
                                                         self.G * self.Hkv, self.Hkv, top),), 0xFF,
                            dtype=torch.uint8, device="cuda")
        tq.tq_chunk_attention(self.c, max_seq_len=top, out=out, workspace=ws, scale=scale, Hkv=self.Hkv, **args)
        return out

    def check(self, out, label, scale=0.0, only=None, skip=None, heads=None):
        import torch
        at, worst, got2, may2 = 0, 0.0, 0.0, 0.0
        hs = range(self.G * self.Hkv) if heads is None else heads
        for b, (n, L) in enumerate(zip(self.nq, self.lens)):
            if n and (only is None or b in only):
                for h in hs:
                    hk = slice(h // self.G, h // self.G + 1)
                    o, A, e, V = attend64(self.q[at:at + n, h:h + 1].double(), self.K[b][:, hk], self.V[b][:, hk], L - n, scale,
                                          self.kerr[b][:, hk], self.verr[b][:, hk], None if skip is None else skip.get(b))
                    bd = bound(o, A, e, V, L, float(self.V[b].abs().max()), out.dtype == torch.float16)
                    err = (out[at:at + n, h:h + 1].double() - o).abs()
                    worst = max(worst, float((err / bd.clamp_min(1e-30)).max()))
                    got2 += float(err.square().sum())
                    may2 += float(rms_bound(A, self.q[at:at + n, h:h + 1].double(), self.K[b][:, hk], 1, scale).square().sum())
                    assert bool((err <= bd).all()), (label, b, h, n, L, float((err / bd).max()), int((err > bd).sum()))
            at += n
        record(label, {"max_err_over_bound": worst, "rms_over_bound": math.sqrt(got2 / max(may2, 1e-30))})
        assert got2 <= may2, (label, math.sqrt(got2 / may2))


@pytest.mark.parametrize("nq,ctx,G,Hkv,bits,rot,km,fp32", [
    ([1], [1], 1, 1, 4, 0, 0, True), ([1], [16], 4, 2, 4, 1, 0, True), ([3], [17], 1, 1, 4, 0, 0, False),
    ([1], [128], 2, 1, 3, 0, 0, True), ([2], [129], 3, 1, 2, 0, 0, True), ([5], [257], 8, 1, 4, 0, 1, True),
    ([4, 4, 4, 4], [1000, 513, 2047, 16], 4, 2, 4, 0, 0, False), ([16, 100], [300, 777], 1, 2, 2, 1, 1, True),
    ([1, 1, 70, 1, 33, 1], [301, 77, 190, 409, 33, 1], 4, 2, 3, 0, 0, True), ([0, 5, 0], [40, 60, 0], 5, 1, 3, 1, 1, True),
    ([200], [200], 4, 1, 4, 1, 1, True), ([300], [700], 7, 1, 4, 0, 0, True), ([64], [4096], 8, 2, 2, 1, 0, False),
    ([1, 2, 3], [5000, 130, 3], 16, 1, 4, 0, 0, True), ([9], [640], 128, 1, 4, 0, 0, True), ([40], [333], 100, 1, 3, 0, 1, True)])
def test_chunk(orc, nq, ctx, G, Hkv, bits, rot, km, fp32):
    c = Case(orc, nq, ctx, G, Hkv, bits, rot, km, seed=sum(ctx))
    out = c.run(fp32)
    assert _tq().tq_get_device_error(c.c) == 0
    c.check(out, "chunk %s of %s G%d b%d rot%d km%d" % (nq, ctx, G, bits, rot, km))


def test_chunk_many_sequences(orc):
    r = random.Random(3)
    ctx = [r.choice([1, 5, 16, 31, 128, 129, 300]) for _ in range(70)]
    nq = [min(n, r.choice([0, 1, 1, 2, 5, 40])) for n in ctx]
    c = Case(orc, nq, ctx, 4, 2, seed=8)
    out = c.run()
    assert _tq().tq_get_device_error(c.c) == 0
    c.check(out, "chunk 70 sequences", heads=[0, 5])


@pytest.mark.parametrize("nq,G", [(1, 4), (40, 4), (300, 2)])
def test_chunk_long_context_and_loud_queries(orc, nq, G):
    """The tokens split over CTAs; scores far apart, so that splits' maxima differ."""
    c = Case(orc, [nq], [20011], G, 1, seed=4, loud=12.0)
    out = c.run()
    assert _tq().tq_get_device_error(c.c) == 0
    c.check(out, "chunk %d of 20011 G%d loud" % (nq, G))


def test_chunk_scale_and_larger_bound(orc):
    """A softmax scale of one's own; max_seq_len far above the lengths."""
    c = Case(orc, [7, 2], [300, 90], 4, 2, seed=5)
    c.check(c.run(top=4000, scale=0.5), "chunk scale 0.5", scale=0.5)


def test_chunk_agrees_with_prefill_and_decode(orc):
    """The one-sequence prefill and the decode see the same tokens: within both bars."""
    import torch
    tq = _tq()
    c = Case(orc, [33], [233], 4, 2, seed=6)
    got = c.run()
    c.check(got, "chunk 33 of 233")
    pre = torch.empty_like(got)
    tq.tq_prefill_attention(c.c, c.q, c.kc, c.vc, c.bt[0].contiguous(), 200, pre, Hkv=2)
    assert float((pre - got).abs().max()) <= 2 * (2e-3 + 2.0 ** -10 * float(c.V[0].abs().max()))


def test_chunk_bad_pages_and_lengths(orc):
    """A block id out of range: its page is skipped.  A length that cannot be: zero rows, the
    other sequences untouched by it."""
    import torch
    tq = _tq()
    c = Case(orc, [6, 20], [150, 400], 4, 2, seed=7)
    ref = c.run()
    for bad in (10 ** 6, -1, c.kc.shape[0]):
        bt = c.bt.clone()
        bt[1, 3] = bad
        out = c.run(block_table=bt)
        assert tq.tq_get_device_error(c.c) == tq.DEVERR_BLOCK
        assert torch.equal(out[:6], ref[:6])
        skip = torch.zeros(400, dtype=torch.bool, device="cuda")
        skip[48:64] = True
        c.check(out, "chunk page skipped", only=[1], skip={1: skip})
    # every page bad: nothing to attend, zero rows
    out = c.run(block_table=torch.where(torch.arange(2, device="cuda")[:, None] == 1, -1, c.bt))
    assert tq.tq_get_device_error(c.c) == tq.DEVERR_BLOCK
    assert torch.equal(out[:6], ref[:6]) and bool((out[6:] == 0).all())
    for L in ([150, 19], [150, -3], [150, 10 ** 6], [150, c.max_blocks * 16 + 1]):
        out = c.run(seq_lens=torch.tensor(L, dtype=torch.int32, device="cuda"), top=600)
        assert tq.tq_get_device_error(c.c) == tq.DEVERR_SEQLEN, L
        assert bool((out[6:] == 0).all()) and bool(torch.isfinite(out[:6]).all())
        c.check(out, "chunk beside a bad length", only=[0])
    out = c.run(top=300)  # longer than max_seq_len says
    assert tq.tq_get_device_error(c.c) == tq.DEVERR_SEQLEN and bool((out[6:] == 0).all())
    for cu in ([0, 30, 26], [0, 6, 27], [-1, 6, 26]):
        c.run(cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert tq.tq_get_device_error(c.c) & tq.DEVERR_SEQLEN


@pytest.mark.parametrize("nq,G", [(6, 4), (30, 4), (150, 4)])
@pytest.mark.parametrize("val", [float("nan"), float("inf")])
def test_chunk_norms_that_are_not_finite(orc, nq, G, val):
    """A norm that is not finite, of a token among the new ones: the queries before it equal the
    run without it to the bit, those from it on are not finite (a rotated value reaches every
    coordinate); a bad gamma or key norm likewise."""
    import torch
    tq = _tq()
    L, at = 300, 300 - nq // 2
    c = Case(orc, [nq, 2], [L, 40], G, 1, seed=14)
    ref = c.run()
    slot = int(c.slots[0][at])
    keep = c.kc.clone(), c.vc.clone()
    for cache, off in ((c.vc, 16 * 64), (c.kc, 16 * 80), (c.kc, 16 * 84)):
        cache[slot // 16, 0].view(torch.float32)[off // 4 + slot % 16] = val
        out = c.run()
        assert tq.tq_get_device_error(c.c) == 0
        first = at - (L - nq)
        assert torch.equal(out[:first], ref[:first]) and torch.equal(out[nq:], ref[nq:])
        # (an infinite key scalar times a negative product is a score of -inf: weight 0, a finite row)
        if cache is c.vc or math.isnan(val):
            assert not bool(torch.isfinite(out[first:nq]).any())
        c.kc.copy_(keep[0])
        c.vc.copy_(keep[1])


def test_chunk_rows_outside_and_empty_calls(orc):
    import torch
    tq = _tq()
    c = Case(orc, [6, 20], [150, 400], 4, 2, seed=9)
    ref = c.run()
    big = torch.cat([c.q[:3], c.q, c.q[:5]])
    out = torch.full(big.shape, 7.0, device="cuda")
    c.run(q=big, cu_q=c.cu + 3, out=out)
    assert tq.tq_get_device_error(c.c) == 0
    assert torch.equal(out[3:29], ref) and bool((out[:3] == 7).all()) and bool((out[29:] == 7).all())
    n0 = tq.tq_launch_count()
    c.run(q=c.q[:0], cu_q=torch.zeros(3, dtype=torch.int32, device="cuda"), out=out[:0],
          ws=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    assert tq.tq_launch_count() == n0
    need = tq.tq_chunk_workspace_bytes(c.c, 2, 26, 8, 2, 400)
    for bad in (dict(ws=torch.empty(need - 1, dtype=torch.uint8, device="cuda")), dict(scale=-1.0),
                dict(scale=float("nan")), dict(out=c.q), dict(k_cache=c.kc[:0], v_cache=c.vc[:0])):
        with pytest.raises(tq.TQError) as e:
            c.run(**bad)
        assert e.value.status == tq.TQ_ERR_INVALID_ARG
    assert tq._lib.tq_chunk_workspace_bytes(c.c.handle, 0, 1, 8, 2, 16) == 0
    assert tq._lib.tq_chunk_workspace_bytes(c.c.handle, 1, 1, 7, 2, 16) == 0
    assert tq._lib.tq_chunk_workspace_bytes(c.c.handle, 1, 1, 258, 2, 16) == 0
    assert tq._lib.tq_chunk_workspace_bytes(c.c.handle, 1, -1, 8, 2, 16) == 0
    assert tq._lib.tq_chunk_workspace_bytes(c.c.handle, 65536, 1, 8, 2, 1 << 20) == 0  # 2^36 rows


def test_chunk_same_block_twice(orc):
    """Two sequences that share their pages (a common prefix), and one page used twice."""
    import torch
    c = Case(orc, [6, 6], [150, 150], 4, 2, seed=10)
    bt = c.bt.clone()
    bt[1] = bt[0]
    q = torch.cat([c.q[:6], c.q[:6]])
    out = c.run(q=q, block_table=bt)
    assert torch.equal(out[:6], out[6:])
    bt[0, 1] = bt[0, 0]
    out = c.run(block_table=bt)
    c.K[0][16:32], c.V[0][16:32] = c.K[0][:16], c.V[0][:16]
    c.kerr[0][16:32], c.verr[0][16:32] = c.kerr[0][:16], c.verr[0][:16]
    c.check(out, "chunk one page twice", only=[0])


def test_chunk_streams_graphs_and_repeats(orc):
    import torch
    tq = _tq()
    c = Case(orc, [1, 30, 9], [900, 77, 3000], 4, 2, seed=11)
    ref = c.run(fp32=False)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs, spaces = [torch.zeros_like(ref) for _ in range(6)], []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        spaces.append(torch.empty(tq.tq_chunk_workspace_bytes(c.c, 3, 40, 8, 2, 3000), dtype=torch.uint8, device="cuda"))
    for i, o in enumerate(outs):
        with torch.cuda.stream(streams[i % 3]):
            c.run(out=o, ws=spaces[i % 3])
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    out = torch.zeros_like(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(out=out, ws=spaces[0])
    c.q.mul_(0.5)
    c.L.copy_(torch.tensor([500, 77, 2111], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, c.run(fp32=False)) and tq.tq_get_device_error(c.c) == 0


def test_rope_prompt_compress_chunk_together(orc):
    """A prompt through the whole path: fused projection -> rotary positions -> prompt
    attention and compress -> more tokens, rotated and compressed -> chunk attention -> one
    token by the decode.  The chunk equals the prompt attention over the decompressed cache."""
    import torch
    tq = _tq()
    Hq, Hkv, lens, more, nb = 8, 2, [130, 47], [20, 5], 32
    ctx = gpu_ctx(4, 31, 0, 0)
    o = orc.Oracle(128, 4, 31)
    table = tq.tq_rope_plan(128, tq.ROPE_HALF, 500000.0, tq.ROPE_SCALE_YARN, 4.0, 8192, 1.0, 32.0)
    g = torch.Generator(device="cuda").manual_seed(12)
    kc = torch.zeros((nb, Hkv, tq.tq_chunk_bytes(ctx, 0)), dtype=torch.uint8, device="cuda")
    vc = torch.zeros((nb, Hkv, tq.tq_chunk_bytes(ctx, 1)), dtype=torch.uint8, device="cuda")
    bt = torch.randperm(nb, generator=g, device="cuda").to(torch.int32).view(2, 16)
    done = [0, 0]

    def step(ns):
        T = sum(ns)
        x = torch.randn((T, (Hq + 2 * Hkv) * 128), generator=g, device="cuda").half()
        q, k = x[:, :Hq * 128].view(T, Hq, 128), x[:, Hq * 128:(Hq + Hkv) * 128].view(T, Hkv, 128)
        v = x[:, (Hq + Hkv) * 128:].view(T, Hkv, 128)
        pos = torch.cat([torch.arange(d, d + n) for d, n in zip(done, ns)]).to("cuda", torch.int32)
        seq = torch.cat([torch.full((n,), b) for b, n in enumerate(ns)]).cuda()
        qr, kr = torch.empty((T, Hq, 128), dtype=torch.float16, device="cuda"), torch.empty((T, Hkv, 128), dtype=torch.float16, device="cuda")
        tq.tq_rope(table, q, k, pos, qr, kr)
        slots = (bt[seq, pos.long() // 16] * 16 + pos % 16).to(torch.int32)
        tq.tq_compress(ctx, kr, v.contiguous(), slots, kc, vc)
        for b, n in enumerate(ns):
            done[b] += n
        cu = torch.tensor([0] + list(np.cumsum(ns)), dtype=torch.int32, device="cuda")
        return qr, kr, v, cu

    q, k, v, cu = step(lens)
    first = torch.empty((sum(lens), Hq, 128), dtype=torch.float16, device="cuda")
    tq.tq_prompt_attention(ctx, q, k, v, cu, first)
    at = 0
    for n in lens:
        w, A, e, V = attend64(q[at:at + n].double(), k[at:at + n].double(), v[at:at + n].double(), 0)
        assert bool(((first[at:at + n].double() - w).abs() <= bound(w, A, e, V, n, float(v.abs().max()), True)).all())
        at += n
    for ns in (more, [1, 1]):
        q, _, _, cu = step(ns)
        L = torch.tensor(done, dtype=torch.int32, device="cuda")
        out = torch.empty((sum(ns), Hq, 128), dtype=torch.float16, device="cuda")
        ws = torch.empty(tq.tq_chunk_workspace_bytes(ctx, 2, sum(ns), Hq, Hkv, 160), dtype=torch.uint8, device="cuda")
        tq.tq_chunk_attention(ctx, q, cu, kc, vc, bt, L, 160, out, ws)
        kn, vn, btn = kc.cpu().numpy(), vc.cpu().numpy(), bt.cpu().numpy()
        kz = kn.copy()
        kz[..., -64:] = 0
        at = 0
        for b, n in enumerate(ns):
            t = np.arange(done[b])
            sl = (btn[b][t // 16] * 16 + t % 16).astype(np.int32)
            K, Vv, Kz = (torch.as_tensor(o.decompress_paged(kind, c, sl, Hkv), device="cuda")
                         for kind, c in ((0, kn), (1, vn), (0, kz)))
            w, A, e, V = attend64(q[at:at + n].double(), K, Vv, done[b] - n, None, 2 * U16 * Kz.norm(dim=2), 2 * U16 * Vv.norm(dim=2))
            b_ = bound(w, A, e, V, done[b], float(Vv.abs().max()), True)
            assert bool(((out[at:at + n].double() - w).abs() <= b_).all())
            at += n
    dec = torch.empty((2, Hq, 128), dtype=torch.float16, device="cuda")
    ws = torch.empty(tq.tq_decode_workspace_bytes(ctx, 2, Hq, Hkv, 160), dtype=torch.uint8, device="cuda")
    tq.tq_decode_attention(ctx, q, kc, vc, bt, L, 160, dec, ws)
    assert float((dec.float() - out.float()).abs().max()) <= 2 * (2e-3 + 2.0 ** -10 * 6)
    assert tq.tq_get_device_error(ctx) == 0
