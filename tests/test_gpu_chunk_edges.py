"""Edges of tq_chunk_attention and tq_prompt_attention: what test_gpu_chunk.py and
test_gpu_prompt.py do not reach (bounds: attention64.py)."""
import math

import numpy as np
import pytest

from attention64 import U16, attend64, rms_bound
from parity import gpu_ctx
from test_gpu_chunk import Case

pytestmark = pytest.mark.gpu

# (queries, query heads of a group) for the three ways of a chunk: up to 32 and up to 128 rows a
# sequence straight over the pages, more of them after a decompression
WAYS = [(1, 4), (8, 4), (30, 4), (150, 4)]


def _tq():
    from kv_cache_vector_02_b200 import tq
    return tq


def _scalars(c):
    """Views of a case's key norms, key gammas (None without a sketch) and value norms: [blocks, Hkv, 16]."""
    import torch
    k, v = c.kc.view(torch.float32), c.vc.view(torch.float32)
    if c.c.key_mode == 0:
        return k[..., -32:-16], k[..., -16:], v[..., -16:]
    return k[..., -16:], None, v[..., -16:]


def _refresh(c, orc):
    """The case's 64-bit keys and values again, from its caches as they are now."""
    import torch
    o = orc.Oracle(128, c.c.bits, c.c.seed, rot=c.c.rotation, key_mode=c.c.key_mode)
    kc, vc = c.kc.cpu().numpy(), c.vc.cpu().numpy()
    kz = kc.copy()
    if c.c.key_mode == 0:
        kz[..., -64:] = 0
    K, V, Kz = ([torch.as_tensor(o.decompress_paged(kind, cache, s, c.Hkv), device="cuda") for s in c.slots]
                for kind, cache in ((0, kc), (1, vc), (0, kz)))
    c.K, c.V = K, V
    c.kerr, c.verr = [2 * U16 * x.norm(dim=2) for x in Kz], [2 * U16 * x.norm(dim=2) for x in V]


@pytest.mark.parametrize("nq,G", WAYS)
def test_starts_and_lengths_far_out_of_range(orc, nq, G):
    """Entries whose differences pass 32 bits: an error, and nothing outside the rows written."""
    import torch
    tq = _tq()
    c = Case(orc, [nq, nq], [300, 300], G, 1, seed=22)
    n = 2 * nq
    v = torch.randn((n, 1, 128), device="cuda").half()
    for cu in ([0, nq, -2 ** 31], [0, nq, -2 ** 31 + nq - 1], [1, 1, -2 ** 31 + 2], [n, -2 ** 31 + 5, 2 ** 31 - 1],
               [0, nq, 2 ** 31 - 1]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        for prompt in (False, True):
            room = torch.full((3 * n, G, 128), 7.0, device="cuda")
            out = room[n:2 * n]
            if prompt:
                tq.tq_prompt_attention(c.c, c.q, v, v, cu, out)
            else:
                c.run(cu_q=cu, out=out)
            assert tq.tq_get_device_error(c.c) & tq.DEVERR_SEQLEN
            assert bool((room[:n] == 7).all()) and bool((room[2 * n:] == 7).all())
    ref = c.run()
    for L in (-2 ** 31, -2 ** 31 + nq - 1, 2 ** 31 - 1):
        out = c.run(seq_lens=torch.tensor([300, L], dtype=torch.int32, device="cuda"))
        assert tq.tq_get_device_error(c.c) == tq.DEVERR_SEQLEN
        assert torch.equal(out[:nq], ref[:nq]) and not bool(out[nq:].any())


@pytest.mark.parametrize("nq,G", WAYS)
def test_zero_values_count_in_the_softmax(orc, nq, G):
    """Tokens whose values are 0 weigh as any: one token of large values, and thousands of zero
    ones 13.5 (base 2) below its score that carry a quarter of the weight."""
    c = Case(orc, [nq], [4096], G, 1, seed=20)
    kn, kg, vn = _scalars(c)
    page, r = int(c.slots[0][5]) // 16, 5
    for x in (kn, kg, vn):
        x.zero_()
    kn[page, 0, r], vn[page, 0, r] = 4.0, 2.0 ** 13 * math.sqrt(128)
    _refresh(c, orc)
    key = c.K[0][5, 0]
    c.q[:] = (key / key.norm() * 3).half()
    scale = 13.5 * math.log(2.0) / float(c.q[0, 0].double() @ key)
    c.check(c.run(scale=scale), "chunk zero values %d" % nq, scale=scale)
    vn.zero_()
    assert not bool(c.run(scale=scale).any())
    # among ordinary ones
    c = Case(orc, [nq], [700], G, 1, seed=21)
    _scalars(c)[2][:, :, ::3] = 0.0
    _refresh(c, orc)
    c.check(c.run(), "chunk some zero values %d" % nq)


@pytest.mark.parametrize("nq,G", WAYS)
@pytest.mark.parametrize("rot,km", [(0, 0), (1, 0), (1, 1)])
def test_queries_of_any_fp16_size(orc, nq, G, rot, km):
    """Queries whose rotation or sketch lies beyond fp16: along a row of the sketch matrix and a
    column of the rotation, beside ordinary and tiny ones."""
    import torch
    tq = _tq()
    c = Case(orc, [nq, 3], [400, 90], G, 1, rot=rot, km=km, seed=23)
    P = tq.tq_export_params(c.c)
    S, R = torch.as_tensor(P["S"], device="cuda").double(), torch.as_tensor(P["R"], device="cuda").double()
    loud = [S[3] * 500, S[7] * 60000, -S[9] * 2000, R[:, 5] * (60000 / R[:, 5].abs().max()), R[:, 0] * 5e4]
    for i in range(min(nq * G, 40)):
        if i % 6 < 5:
            c.q[i // G, i % G] = loud[i % 6].half()
        else:
            c.q[i // G, i % G] *= 2.0 ** -8
    assert bool(torch.isfinite(c.q).all())
    # (scores of the loudest: 60000 sqrt(128) * |k| / sqrt(128) at random angles, times the scale)
    scale = 2e-6
    out = c.run(scale=scale)
    assert bool(torch.isfinite(out).all())
    c.check(out, "chunk loud queries %d" % nq, scale=scale)
    # a query that is not finite reaches its own head's row only
    c.q[0, 1] = float("inf")
    bad = c.run(scale=scale)
    keep = torch.ones(bad.shape[:2], dtype=torch.bool, device="cuda")
    keep[0, 1] = False
    assert torch.equal(bad[keep], out[keep]) and bool(torch.isnan(bad[0, 1]).all())


@pytest.mark.parametrize("nq,G", WAYS)
def test_outputs_and_workspaces_over_inputs(orc, nq, G):
    """An output or a workspace over a list or a cache is refused, and the input stays as it was."""
    import torch
    tq = _tq()
    c = Case(orc, [nq], [300], G, 1, seed=24)
    need = tq.tq_chunk_workspace_bytes(c.c, 1, nq, G, 1, 300)
    room = torch.zeros(need + (1 << 20), dtype=torch.uint8, device="cuda")
    out = torch.empty(c.q.shape, dtype=torch.float32, device="cuda")

    def inside(t, at):
        """A copy of t in `room`, `at` bytes from its start."""
        n = t.numel() * t.element_size()
        view = room[at:at + n].view(t.dtype).view(t.shape)
        view.copy_(t)
        return view

    n_out = out.numel() * 4
    for name in ("cu_q", "seq_lens", "block_table", "k_cache", "v_cache"):
        t = dict(cu_q=c.cu, seq_lens=c.L, block_table=c.bt, k_cache=c.kc, v_cache=c.vc)[name]
        for at, kw in ((0, dict(ws=room[:need])), (need - 16, dict(ws=room[:need])),
                       (0, dict(out=room[:n_out].view(torch.float32).view(out.shape))),
                       (n_out - 16, dict(out=room[:n_out].view(torch.float32).view(out.shape)))):
            view = inside(t, at)
            n0 = tq.tq_launch_count()
            with pytest.raises(tq.TQError) as e:
                c.run(**{name: view}, **kw)
            assert e.value.status == tq.TQ_ERR_INVALID_ARG and tq.tq_launch_count() == n0, (name, at)
            assert torch.equal(view, t)
        # right behind a workspace and an output: allowed
        behind = -(-max(need, n_out) // 256) * 256
        c.check(c.run(ws=room[:need], **{name: inside(t, behind)}), "chunk %s behind the workspace" % name)
        o = room[:n_out].view(torch.float32).view(out.shape)
        c.check(c.run(out=o, **{name: inside(t, behind)}), "chunk %s behind the output" % name)


def test_lengths_next_to_31_bits():
    """Token numbers a few tiles past the longest sequence stay within 32 bits."""
    tq = _tq()
    c = gpu_ctx()
    for top in (2 ** 31 - 1, 2 ** 31 - 200, 2 ** 31 - 1024):
        assert tq._lib.tq_chunk_workspace_bytes(c.handle, 1, 1, 1, 1, top) == 0, top
    assert tq._lib.tq_chunk_workspace_bytes(c.handle, 1, 1, 1, 1, 2 ** 31 - 4096) > 0


def test_one_workspace_for_smaller_calls(orc):
    """A workspace sized for the largest step takes every step of as many sequences with fewer
    queries or a smaller bound on the lengths, whatever way and split those would choose."""
    import torch
    tq = _tq()
    for B, G, Hkv, most, top in ((1, 4, 2, 900, 4096), (2, 4, 1, 300, 1000), (1, 1, 1, 400, 256), (3, 8, 1, 200, 100)):
        c = Case(orc, [1] * B, [top - 7 * b for b in range(B)], G, Hkv, seed=25)
        g = torch.Generator(device="cuda").manual_seed(26)
        ws = torch.full((tq.tq_chunk_workspace_bytes(c.c, B, most, G * Hkv, Hkv, top),), 0xFF, dtype=torch.uint8, device="cuda")
        n = most
        while n >= 1:
            left = min(n, top - 7 * B)
            c.nq = [left] + [min(n - left, 40)] * (B > 1) + [0] * (B - 2)
            c.cu = torch.tensor([0] + list(np.cumsum(c.nq)), dtype=torch.int32, device="cuda")
            c.q = (torch.randn((sum(c.nq), G * Hkv, 128), generator=g, device="cuda") / math.sqrt(128)).half()
            assert tq.tq_chunk_workspace_bytes(c.c, B, n, G * Hkv, Hkv, top) > 0
            out = c.run(ws=ws)
            assert tq.tq_get_device_error(c.c) == 0
            c.check(out, "chunk %d queries in a workspace for %d" % (n, most), heads=[0, G * Hkv - 1])
            n = n * 2 // 3
        # a smaller bound on the lengths
        short = min(top, 90)
        s = Case(orc, [2] * B, [short - b for b in range(B)], G, Hkv, seed=27)
        s.check(s.run(ws=ws), "chunk short sequences in a workspace for long ones")
    # and more than a pass of heads: half the bound fits more heads a pass than the whole one
    c = gpu_ctx()
    big = tq.tq_chunk_workspace_bytes(c, 1, 600, 6, 3, 1200000)
    s = Case(orc, [300], [700], 2, 3, seed=28)
    s.check(s.run(top=600000, ws=torch.empty(big, dtype=torch.uint8, device="cuda")), "chunk fewer heads a pass")


@pytest.mark.parametrize("nq,G", WAYS)
def test_many_small_weights_add_up(orc, nq, G):
    """131072 tokens of weight 2^-26 beside one of weight 1: 0.2 % of the output, all of one sign.
    Bound on the output's share along the small ones' value w, with o = u (the dominant token's
    value) as the accumulator holds it, |u| |w| / |w|^2 of it along w:
      * u's roundings: 2^-11 of it;
      * the accumulator: an MMA adds 16 tokens, L / 16 additions, each truncated by up to 2^-23 of it;
      * the sum that the output is divided by: at most L / 4 additions to the accumulator that
        holds the large weight, each off by 2^-24 of it, times the output;
      * the small weights: the score's error, and 2^-32 for each below P's least step.
    Together two thirds of what the small weights give."""
    import torch
    L = 131072
    # (as many CTAs as SMs, so that no sequence is split: a split without the first token has no small weights)
    B, Hkv = (37, 4) if nq * G <= 128 else (1, 1)
    c = Case(orc, [1], [32], G, Hkv, seed=29, spare=0)
    kn, kg, vn = _scalars(c)
    kn.zero_(), kg.zero_()
    first, rest = (int(c.slots[0][t]) // 16 for t in (0, 16))
    code, (vc0, vc1) = 64, (c.vc[first, 0], c.vc[rest, 0])
    # one value for every small token, another of the same norm for the dominant one
    for page in (vc0, vc1):
        page[:16 * code] = page[:16 * code].view(16, code)[3].repeat(16)
    vc0[code:16 * code] = vc1[code:16 * code]
    vn[:] = 30.0
    kn[first, 0, 0] = 4.0
    c.kc[:], c.vc[:] = c.kc[:, :1].clone(), c.vc[:, :1].clone()  # every head alike
    _refresh(c, orc)
    u, w, key = c.V[0][0, 0], c.V[0][1, 0], c.K[0][0, 0]
    c.bt = torch.full((B, L // 16), rest, dtype=torch.int32, device="cuda")
    c.bt[:, 0] = first
    c.top = L
    c.L = torch.full((B,), L, dtype=torch.int32, device="cuda")
    c.cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * nq
    c.q = torch.empty((B * nq, G * Hkv, 128), dtype=torch.float16, device="cuda")
    c.q[:] = (key / key.norm() * 3).half()
    scale = 26 * math.log(2.0) / float(c.q[0, 0].double() @ key)
    out = c.run(scale=scale).double()
    small = (L - nq + torch.arange(nq, device="cuda")).repeat(B).double() * 2.0 ** -26  # all that each query sees but the first token
    share = out @ w / (w @ w)
    want = (float(u @ w / (w @ w)) + small) / (1 + small)
    # (the score's error moves the small weights: 26 ln 2 times the bound of its rounding)
    tol = (U16 + L / 16 * 2.0 ** -23) * float(u.abs() @ w.abs() / (w @ w)) + small * 26 * 4 * U16 + L * 2.0 ** -32
    tol = tol + L / 4 * 2.0 ** -24 * want.abs()
    assert bool((tol < 0.75 * small).all())
    assert bool(((share - want[:, None]).abs() <= tol[:, None]).all()), float((share - want[:, None]).abs().max())


def test_many_small_weights_add_up_prompt():
    """The same over a prompt's exact values: a coordinate that the dominant token lacks."""
    import torch
    tq = _tq()
    T = 30000
    q, k = (torch.zeros((T, 1, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    v = torch.ones_like(k)
    q[:, 0, 0], k[0, 0, 0], v[0, 0, 5] = 4.0, 4.0, 0.0
    out = torch.empty((T, 1, 128), device="cuda")
    tq.tq_prompt_attention(gpu_ctx(), q, k, v, torch.tensor([0, T], dtype=torch.int32, device="cuda"), out,
                           scale=26 * math.log(2.0) / 16)
    small = torch.arange(T, device="cuda").double() * 2.0 ** -26
    want = small / (1 + small)
    # the scale and the exponent's argument in fp32 (26 ln 2 each off by 2^-22), P in fp16 (its least step 2^-32)
    tol = small * (26 * 2.0 ** -21 + U16) + T * 2.0 ** -33
    err = (out[:, 0, 5].double() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("nq,G", WAYS)
def test_values_beyond_fp16_reach_their_queries_only(orc, nq, G):
    """A value norm whose coordinates pass fp16, of a token among the new ones: the queries before
    it equal the run without it to the bit."""
    import torch
    c = Case(orc, [max(nq, 4), 2], [300, 40], G, 1, seed=30)
    n = c.nq[0]
    at = 300 - n // 2
    ref = c.run()
    vn = _scalars(c)[2]
    slot = int(c.slots[0][at])
    for norm in (2.0 ** 15 * math.sqrt(128), 2.0 ** 20, 1e38):
        vn[slot // 16, 0, slot % 16] = norm
        out = c.run()
        first = at - (300 - n)
        assert torch.equal(out[:first], ref[:first]) and torch.equal(out[n:], ref[n:])


@pytest.mark.parametrize("nq,G", WAYS)
def test_sequences_without_queries_are_not_looked_at(orc, nq, G):
    """A batch filled up with empty sequences whose lengths and pages are left over."""
    import torch
    tq = _tq()
    n = 4 * nq  # (the rows of a sequence on average choose the way)
    c = Case(orc, [0, n, 0, 0], [40, 700, 90, 200], G, 2, seed=40)
    ref = c.run()
    c.check(ref, "chunk beside empty sequences")
    bt = c.bt.clone()
    bt[0], bt[2], bt[3] = -1, 10 ** 6, -5
    for L in ([40, 700, 90, 200], [-7, 700, 10 ** 6, 704]):
        out = c.run(block_table=bt, seq_lens=torch.tensor(L, dtype=torch.int32, device="cuda"))
        assert tq.tq_get_device_error(c.c) == 0
        assert torch.equal(out, ref)


@pytest.mark.parametrize("bits,km", [(4, 0), (3, 0), (2, 0), (4, 1), (3, 1), (2, 1)])
@pytest.mark.parametrize("nq,G", WAYS)
def test_every_width_on_every_way(orc, nq, G, bits, km):
    c = Case(orc, [nq, 2], [400, 33], G, 2, bits, nq % 2, km, seed=31)
    out = c.run()
    assert _tq().tq_get_device_error(c.c) == 0
    c.check(out, "chunk %d bits, mode %d, %d x %d rows" % (bits, km, nq, G))


@pytest.mark.parametrize("B", [4, 12, 25, 40])
def test_every_shape_of_the_join(orc, B):
    """256, 768, 1600 and 2560 rows, the tokens split and not."""
    c = Case(orc, [2] * B, [130 + 50 * (b % 5) for b in range(B)], 4, 8, seed=32)
    c.check(c.run(), "chunk join of %d rows" % (64 * B), heads=[0, 13, 31])


@pytest.mark.parametrize("nq,G,top,groups,split", [(300, 2, 800000, 2, True), (300, 2, 1200000, 3, True),
                                                   (148, 128, 800000, 2, False)])
def test_heads_in_passes(orc, nq, G, top, groups, split):
    """More decompressed tokens than are held at a time, by the bound on the lengths: the kv heads
    go in passes (2 + 1 and 1 + 1 + 1), with their tokens split over CTAs and not."""
    import torch
    tq = _tq()
    c = Case(orc, [nq], [nq + 60], G, 3, seed=33)
    n0 = tq.tq_launch_count()
    out = c.run(top=top)
    assert tq.tq_launch_count() - n0 == groups * (3 if split else 2)
    assert tq.tq_get_device_error(c.c) == 0
    c.check(out, "chunk heads in %d passes, G %d" % (groups, G))
    bt = c.bt.clone()
    bt[0, 1] = -1
    skip = torch.zeros(nq + 60, dtype=torch.bool, device="cuda")
    skip[16:32] = True
    out = c.run(top=top, block_table=bt)
    assert tq.tq_get_device_error(c.c) == tq.DEVERR_BLOCK
    c.check(out, "chunk heads in passes, a page skipped", skip={0: skip})


@pytest.mark.parametrize("nq,G", WAYS + [(300, 2)])
def test_every_token_once_in_long_contexts(orc, nq, G):
    """Each (query, head) looks at two tokens alone, out of 20011: its own, the last it may see,
    and one at a border of tiles, both with a score of 25; the token behind its own would have 30.
    A token left out, let in or counted twice moves an output by a sixth of
    the two values' difference or more; the bound is six times the root mean square that
    independent roundings give (attention64.py), about 4 % of a value."""
    import torch
    L = 20011
    c = Case(orc, [nq], [L], G, 1, seed=34)
    K, V = c.K[0][:, 0], c.V[0][:, 0]
    own = L - nq + torch.arange(nq, device="cuda")
    borders = torch.tensor([0, 127, 128, 255, 256, 639, 640, 1279, 1280, 2559, 2560, 5119, 5120, 10239, 10240, 19711, 19712],
                           device="cuda")
    behind = (own + 1).clamp(max=L - 1)
    for h in range(G):
        other = own if h == 0 else borders[(torch.arange(nq, device="cuda") * 5 + 3 * h) % len(borders)]
        want = torch.full((nq, 3, 1), 25 * math.sqrt(128), dtype=torch.float64, device="cuda")
        want[:, 2, 0] *= torch.where(own < L - 1, 1.2, 1.0)
        c.q[:, h] = (torch.linalg.pinv(torch.stack([K[own], K[other], K[behind]], 1)) @ want)[..., 0].half()
    out = c.run().double()
    assert _tq().tq_get_device_error(c.c) == 0
    for h in range(G):
        o, A, _, _ = attend64(c.q[:, h:h + 1].double(), c.K[0], c.V[0], L - nq)
        tol = 6 * rms_bound(A, c.q[:, h:h + 1].double(), c.K[0], 1) + L * 2.0 ** -25 * float(V.abs().max())
        err = (out[:, h:h + 1] - o).abs()
        assert bool((err <= tol).all()), (h, float((err / tol).max()))
        # what the bound is worth: one token fewer (for each head's own), and one more, pass it by far
        for first, rows in ((L - nq - 1, slice(None)), (L - nq + 1, slice(0, nq - 1))):
            wrong = attend64(c.q[:, h:h + 1].double(), c.K[0], c.V[0], first)[0]
            assert bool(((wrong - o).abs() > 2 * tol)[rows].flatten(1).any(1).all())
