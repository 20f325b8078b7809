"""tq_prompt_attention against plain attention in 64 bits (bounds: attention64.py)."""
import math

import pytest

from attention64 import attend64, bound, rms_bound
from parity import gpu_ctx, record

pytestmark = pytest.mark.gpu


def _tq():
    from kv_cache_vector_02_b200 import tq
    return tq


def _inputs(T, Hq, Hkv, seed, loud=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (torch.randn((T, Hq, 128), generator=g, device="cuda") * loud).half()
    k = torch.randn((T, Hkv, 128), generator=g, device="cuda").half()
    v = (torch.randn((T, Hkv, 128), generator=g, device="cuda") * 3 + 0.5).half()
    return q, k, v


def _starts(lens, first=0):
    import torch
    c = [first]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def _check(got, q, k, v, lens, label, first=0, scale=0.0, heads=None):
    import torch
    at, worst, got2, may2 = first, 0.0, 0.0, 0.0
    hs = list(range(q.shape[1])) if heads is None else heads
    G = q.shape[1] // k.shape[1]
    for n in lens:
        if n:
            for h in hs:
                sl = slice(at, at + n)
                o, A, e, V = attend64(q[sl, h:h + 1].double(), k[sl, h // G:h // G + 1].double(),
                                   v[sl, h // G:h // G + 1].double(), 0, scale)
                b = bound(o, A, e, V, n, float(v[sl].abs().max()), got.dtype == torch.float16)
                err = (got[sl, h:h + 1].double() - o).abs()
                worst = max(worst, float((err / b).max()))
                got2 += float(err.square().sum())
                may2 += float(rms_bound(A, q[sl, h:h + 1].double(), k[sl, h // G:h // G + 1].double(), 1, scale).square().sum())
                assert bool((err <= b).all()), (label, h, n, float((err / b).max()), int((err > b).sum()))
        at += n
    record(label, {"max_err_over_bound": worst, "rms_over_bound": math.sqrt(got2 / max(may2, 1e-30))})
    assert got2 <= may2, (label, math.sqrt(got2 / may2))


@pytest.mark.parametrize("lens,Hq,Hkv,fp32,loud", [
    ([1], 1, 1, True, 1), ([2], 8, 8, True, 1), ([127], 1, 1, True, 1), ([128], 2, 1, True, 1), ([129], 4, 1, False, 1),
    ([256], 1, 1, True, 1), ([257], 1, 1, True, 4), ([384, 385], 2, 2, True, 1), ([1000], 4, 2, True, 1),
    ([1, 130, 17, 64], 32, 8, False, 1), ([5, 0, 0, 70, 300], 3, 1, True, 1), ([33, 129], 5, 1, True, 1),
    ([200], 7, 1, True, 2), ([50, 260], 16, 1, True, 1), ([300], 40, 1, True, 1), ([40, 3], 128, 1, True, 1),
    ([7, 500], 100, 1, True, 1), ([1024, 640], 16, 2, False, 8), ([2047], 8, 1, True, 1)])
def test_prompt(lens, Hq, Hkv, fp32, loud):
    import torch
    tq = _tq()
    ctx = gpu_ctx()
    T = sum(lens)
    q, k, v = _inputs(T, Hq, Hkv, T + Hq, loud)
    out = torch.full((T, Hq, 128), float("nan"), dtype=torch.float32 if fp32 else torch.float16, device="cuda")
    n0 = tq.tq_launch_count()
    tq.tq_prompt_attention(ctx, q, k, v, _starts(lens), out)
    assert tq.tq_launch_count() == n0 + 1
    assert tq.tq_get_device_error(ctx) == 0
    _check(out, q, k, v, lens, "prompt %s %d/%d" % (lens, Hq, Hkv))


def test_prompt_many_sequences():
    """Hundreds of short sequences (the search for a tile's sequence in several steps)."""
    import random

    import torch
    tq = _tq()
    ctx = gpu_ctx()
    r = random.Random(5)
    lens = [r.choice([0, 1, 2, 3, 31, 33, 64, 90]) for _ in range(1500)]
    T = sum(lens)
    q, k, v = _inputs(T, 4, 1, 9)
    out = torch.full((T, 4, 128), float("nan"), dtype=torch.float32, device="cuda")
    tq.tq_prompt_attention(ctx, q, k, v, _starts(lens), out)
    assert tq.tq_get_device_error(ctx) == 0
    _check(out, q, k, v, lens, "prompt 1500 sequences", heads=[0, 3])


def test_prompt_long_and_scale():
    import torch
    tq = _tq()
    ctx = gpu_ctx()
    lens = [5000, 3333]
    q, k, v = _inputs(sum(lens), 8, 2, 10)
    out = torch.full(q.shape, float("nan"), dtype=torch.float32, device="cuda")
    tq.tq_prompt_attention(ctx, q, k, v, _starts(lens), out, scale=0.3)
    assert tq.tq_get_device_error(ctx) == 0
    _check(out, q, k, v, lens, "prompt long, scale 0.3", scale=0.3, heads=[0, 5])


def test_prompt_rising_scores():
    """Scores that grow along the sequence by far more than the rescale step: the running
    maximum and the accumulator's rescaling carry the result."""
    import torch
    tq = _tq()
    ctx = gpu_ctx()
    n = 900
    q, k, v = _inputs(n, 2, 1, 11)
    q[:, :, 0] = 8.0
    k[:, 0, 0] = torch.linspace(-60, 60, n, device="cuda").half()
    out = torch.full(q.shape, float("nan"), dtype=torch.float32, device="cuda")
    tq.tq_prompt_attention(ctx, q, k, v, _starts([n]), out)
    _check(out, q, k, v, [n], "prompt rising scores")
    k[:, 0, 0] = torch.linspace(60, -60, n, device="cuda").half()
    tq.tq_prompt_attention(ctx, q, k, v, _starts([n]), out)
    _check(out, q, k, v, [n], "prompt falling scores")


def test_prompt_strided_views_and_rows_outside():
    """q, k, v as views into one projection; rows before the first and behind the last
    sequence stay as they were."""
    import torch
    tq = _tq()
    ctx = gpu_ctx()
    T, Hq, Hkv, lens, first = 300, 4, 2, [100, 150], 20
    x = torch.randn((T, (Hq + 2 * Hkv) * 128), device="cuda").half()
    q = x[:, :Hq * 128].view(T, Hq, 128)
    k = x[:, Hq * 128:(Hq + Hkv) * 128].view(T, Hkv, 128)
    v = x[:, (Hq + Hkv) * 128:].view(T, Hkv, 128)
    out = torch.full((T, Hq, 128), 7.0, dtype=torch.float16, device="cuda")
    x[:first] = float("nan")
    x[first + 250:] = float("inf")
    tq.tq_prompt_attention(ctx, q, k, v, _starts(lens, first), out)
    assert tq.tq_get_device_error(ctx) == 0
    assert bool((out[:first] == 7).all()) and bool((out[first + 250:] == 7).all())
    _check(out, q, k, v, lens, "prompt strided", first=first)


@pytest.mark.parametrize("G", [1, 4])
def test_prompt_masked_places_may_hold_anything(G):
    """Non-finite keys and values at one token reach the queries from that token on, and no
    other: the others equal the run without them to the bit."""
    import torch
    tq = _tq()
    ctx = gpu_ctx()
    lens = [200, 333]
    q, k, v = _inputs(sum(lens), G, 1, 12)
    ref = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    tq.tq_prompt_attention(ctx, q, k, v, _starts(lens), ref)
    for tok, what, val in ((150, "v", float("nan")), (199, "v", float("inf")), (40, "k", float("nan")),
                           (200 + 140, "v", float("-inf")), (200 + 130, "k", float("inf")), (200 + 332, "v", float("nan"))):
        k2, v2 = k.clone(), v.clone()
        (v2 if what == "v" else k2)[tok, 0, 17] = val
        out = torch.full(q.shape, 7.0, dtype=torch.float32, device="cuda")
        tq.tq_prompt_attention(ctx, q, k2, v2, _starts(lens), out)
        end = 200 if tok < 200 else 533
        hit = torch.zeros(533, dtype=torch.bool, device="cuda")
        hit[tok:end] = True
        assert torch.equal(out[~hit], ref[~hit]), (tok, what, val)
        if what == "v":  # the value itself, in its column only
            col = out[hit][:, :, 17]
            assert bool((torch.isnan(col) if math.isnan(val) else col == val).all())
            cols = [c for c in range(128) if c != 17]
            assert torch.equal(out[hit][:, :, cols], ref[hit][:, :, cols])
        elif math.isnan(val):
            assert bool(torch.isnan(out[hit]).all())


def test_prompt_bad_lists_and_empty_calls():
    import torch
    tq = _tq()
    ctx = gpu_ctx()
    q, k, v = _inputs(100, 4, 2, 13)
    out = torch.full(q.shape, 7.0, dtype=torch.float32, device="cuda")
    for bad in ([0, 50, 40, 100], [0, 101], [-5, 100], [0, 2 ** 31 - 1]):
        tq.tq_prompt_attention(ctx, q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"), out)
        assert tq.tq_get_device_error(ctx) & tq.DEVERR_SEQLEN, bad
    out.fill_(7.0)
    n0 = tq.tq_launch_count()
    tq.tq_prompt_attention(ctx, q, k, v, torch.zeros(1, dtype=torch.int32, device="cuda"), out)          # B = 0
    tq.tq_prompt_attention(ctx, q[:0], k[:0], v[:0], torch.zeros(3, dtype=torch.int32, device="cuda"), out[:0])
    assert tq.tq_launch_count() == n0
    tq.tq_prompt_attention(ctx, q, k, v, torch.zeros(4, dtype=torch.int32, device="cuda"), out)          # empty sequences
    assert tq.tq_get_device_error(ctx) == 0 and bool((out == 7).all())
    # refusals of the library
    for kw in (dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        with pytest.raises(tq.TQError):
            tq.tq_prompt_attention(ctx, q, k, v, _starts([100]), out, **kw)
    with pytest.raises(tq.TQError):  # 129 query heads per kv head
        qq = torch.zeros((4, 129, 128), dtype=torch.float16, device="cuda")
        tq.tq_prompt_attention(ctx, qq, k[:4, :1], v[:4, :1], _starts([4]), torch.empty_like(qq))
    with pytest.raises(tq.TQError):  # 4 query heads over 3 kv heads
        tq.tq_prompt_attention(ctx, q, q[:, :3], q[:, :3], _starts([100]), out)
    with pytest.raises(tq.TQError):  # output over an input
        tq.tq_prompt_attention(ctx, q, k, v, _starts([100]), q)


def test_prompt_refuses_output_over_the_list():
    import torch
    tq = _tq()
    ctx = gpu_ctx()
    q, k, v = _inputs(8, 2, 1, 15)
    out = torch.zeros_like(q)
    cu = out.view(-1).view(torch.int32)[:2]
    cu.copy_(_starts([8]))
    with pytest.raises(tq.TQError):
        tq.tq_prompt_attention(ctx, q, k, v, cu, out)
    assert cu.tolist() == [0, 8] and not out.view(-1)[4:].any()


def test_prompt_streams_graphs_and_repeats():
    """The same bits on another stream, in a captured and replayed graph, and every time."""
    import torch
    tq = _tq()
    ctx = gpu_ctx()
    lens = [700, 64, 1301]
    q, k, v = _inputs(sum(lens), 8, 2, 14)
    cu = _starts(lens)
    ref = torch.empty_like(q)
    tq.tq_prompt_attention(ctx, q, k, v, cu, ref)
    outs = [torch.zeros_like(q) for _ in range(6)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i, o in enumerate(outs):
        with torch.cuda.stream(streams[i % 3]):
            tq.tq_prompt_attention(ctx, q, k, v, cu, o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    g = torch.cuda.CUDAGraph()
    out = torch.zeros_like(q)
    with torch.cuda.graph(g):
        tq.tq_prompt_attention(ctx, q, k, v, cu, out)
    q.mul_(0.5)
    cu.copy_(_starts([100, 1500, 465]))
    g.replay()
    torch.cuda.synchronize()
    tq.tq_prompt_attention(ctx, q, k, v, cu, ref)
    assert torch.equal(out, ref) and tq.tq_get_device_error(ctx) == 0
