"""tq_rope against the formula in 64 bits.

Bound per value (fp32 arithmetic, one rounding to fp16): the angle is exact to 2^-32 turns
plus its fp32 rounding (pi 2^-25), sincospi is good to 2 ulp, and the two products and their
sum round at 2^-24: (|x1| + |x2|) m 5e-7 in all; then 2^-11 |y| + 2^-25."""
import numpy as np
import pytest

from parity import record

pytestmark = pytest.mark.gpu


def _tq():
    from kv_cache_vector_02_b200 import tq
    return tq


def _want(x, pos, table, sign):
    import torch
    rot, half = table.rot_dim, table.layout == 0
    # the angle from integers: (pos * turns) mod 2^64
    a = np.array([[(int(p) * int(table.turns[i])) % (1 << 64) for i in range(rot // 2)] for p in pos], dtype=np.float64)
    a = torch.as_tensor(a * (2 * np.pi / 2.0 ** 64), device=x.device)[:, None, :] * sign
    y = x.double().clone()
    i = torch.arange(rot // 2, device=x.device)
    i1, i2 = (i, i + rot // 2) if half else (2 * i, 2 * i + 1)
    x1, x2 = y[..., i1].clone(), y[..., i2].clone()
    m = float(table.mscale)
    y[..., i1] = m * (x1 * a.cos() - x2 * a.sin())
    y[..., i2] = m * (x2 * a.cos() + x1 * a.sin())
    slack = torch.zeros_like(y)
    slack[..., i1] = slack[..., i2] = (x1.abs() + x2.abs()) * m * 5e-7
    slack[..., :rot] += 2.0 ** -11 * y[..., :rot].abs() + 2.0 ** -25
    return y, slack


def _check(got, x, pos, table, sign, label):
    y, slack = _want(x, pos, table, sign)
    err = (got.double() - y).abs()
    assert bool((err <= slack).all()), (label, float((err - slack).max()))
    return float((err / slack.clamp_min(1e-30)).max())


def _inputs(T, Hq, Hkv, far, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn((T, Hq, 128), generator=g, device="cuda").half()
    k = (torch.randn((T, Hkv, 128), generator=g, device="cuda") * 20).half()
    pos = torch.randint(0, far, (T,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = far - 1
    pos[-1] = 0
    return q, k, pos


@pytest.mark.parametrize("T,Hq,Hkv,rot,layout,kind,far", [
    (1, 1, 1, 128, 0, 0, 5), (33, 32, 8, 128, 0, 4, 131072), (7, 3, 1, 128, 1, 3, 2 ** 31 - 1), (64, 8, 8, 64, 0, 1, 70000),
    (65, 5, 1, 64, 1, 2, 9000), (19, 2, 2, 20, 0, 0, 9000), (19, 2, 2, 20, 1, 0, 9000), (5, 4, 2, 2, 0, 0, 2 ** 30),
    (5, 4, 2, 2, 1, 0, 2 ** 30), (12, 7, 1, 96, 0, 4, 40000), (12, 7, 1, 98, 1, 1, 40000), (3, 160, 8, 80, 0, 0, 40000),
    (1500, 9, 3, 128, 0, 0, 131072), (2500, 2, 1, 112, 1, 0, 131072)])
def test_rope(T, Hq, Hkv, rot, layout, kind, far):
    import torch
    tq = _tq()
    t = tq.tq_rope_plan(rot, layout, 500000.0, kind, 8.0, 8192, 1.0, 4.0 if kind == 3 else 32.0)
    q, k, pos = _inputs(T, Hq, Hkv, far, T)
    p = pos.cpu().numpy()
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    n0 = tq.tq_launch_count()
    tq.tq_rope(t, q, k, pos, qo, ko)
    assert tq.tq_launch_count() == n0 + 1
    worst = max(_check(qo, q, p, t, 1, "q"), _check(ko, k, p, t, 1, "k"))
    record("rope T%d %d/%d rot%d layout%d scaling%d" % (T, Hq, Hkv, rot, layout, kind), {"max_err_over_bound": worst})
    # in place, and each input alone, give the same bits
    q2, k2 = q.clone(), k.clone()
    tq.tq_rope(t, q2, k2, pos)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    q3 = torch.zeros_like(q)
    tq.tq_rope(t, q, None, pos, q3)
    assert torch.equal(q3, qo)
    k3 = k.clone()
    tq.tq_rope(t, None, k3, pos)
    assert torch.equal(k3, ko)
    # the transposed map
    qt = torch.empty_like(q)
    tq.tq_rope(t, q, None, pos, qt, transpose=True)
    _check(qt, q, p, t, -1, "transposed")


def test_rope_gradient_against_differences():
    """The map is linear: <y(x + d) - y(x), g> = <d, transposed(g)> up to the roundings of the
    three fp16 results (2^-11 of each term's magnitude)."""
    import torch
    tq = _tq()
    t = tq.tq_rope_plan(96, tq.ROPE_HALF, 10000.0, tq.ROPE_SCALE_YARN, 4.0, 2048, 1.0, 32.0)
    q, _, pos = _inputs(40, 4, 1, 60000, 3)
    d = torch.randn_like(q, dtype=torch.float32).half()
    g = torch.randn_like(q, dtype=torch.float32).half()
    y0, y1, gt = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    x1 = (q.double() + d.double()).half()
    tq.tq_rope(t, q, None, pos, y0)
    tq.tq_rope(t, x1, None, pos, y1)
    tq.tq_rope(t, g, None, pos, gt, transpose=True)
    step = x1.double() - q.double()
    left = (y1.double() - y0.double()) * g.double()
    right = step * gt.double()
    tol = ((y1.double().abs() + y0.double().abs()) * g.double().abs() + step.abs() * gt.double().abs()) * (2.0 ** -11 + 1e-6)
    assert bool(((left.sum(-1) - right.sum(-1)).abs() <= tol.sum(-1)).all())


def test_rope_fused_rows_strides_and_skipped_tokens():
    """q and k as views into one projection, outputs with strides of their own; negative
    positions leave rows as they were; the values behind the heads are not touched."""
    import torch
    tq = _tq()
    T, Hq, Hkv = 37, 6, 2
    x = torch.randn((T, (Hq + 2 * Hkv) * 128), device="cuda").half()
    keep = x.clone()
    q, k = x[:, :Hq * 128].view(T, Hq, 128), x[:, Hq * 128:(Hq + Hkv) * 128].view(T, Hkv, 128)
    pos = torch.arange(T, device="cuda", dtype=torch.int32) * 1000
    pos[5] = -1
    pos[36] = -7
    t = tq.tq_rope_plan(64, tq.ROPE_HALF)
    big = torch.full((T, Hq + 3, 128), 7.0, device="cuda").half()
    ko = torch.full((T, Hkv, 128), 7.0, device="cuda").half()
    tq.tq_rope(t, q, k, pos, big[:, :Hq], ko)
    live = pos >= 0
    p = pos.cpu().numpy()
    _check(big[live][:, :Hq], q[live], p[p >= 0], t, 1, "q")
    _check(ko[live], k[live], p[p >= 0], t, 1, "k")
    assert bool((big[~live] == 7).all()) and bool((ko[~live] == 7).all()) and bool((big[:, Hq:] == 7).all())
    tq.tq_rope(t, q, k, pos)  # in place, inside the fused rows
    assert torch.equal(x[~live], keep[~live]) and torch.equal(x[:, (Hq + Hkv) * 128:], keep[:, (Hq + Hkv) * 128:])
    assert torch.equal(q[live], big[live][:, :Hq]) and torch.equal(k[live], ko[live])


def test_rope_non_finite_values_stay_in_their_pair():
    import torch
    tq = _tq()
    t = tq.tq_rope_plan(128, tq.ROPE_INTERLEAVED)
    q = torch.randn((4, 2, 128), device="cuda").half()
    pos = torch.arange(4, device="cuda", dtype=torch.int32)
    a = torch.empty_like(q)
    tq.tq_rope(t, q, None, pos, a)
    q[1, 1, 8] = float("inf")
    b = torch.empty_like(q)
    tq.tq_rope(t, q, None, pos, b)
    same = torch.ones_like(q, dtype=torch.bool)
    same[1, 1, 8:10] = False
    assert torch.equal(a[same], b[same]) and not bool(torch.isfinite(b[1, 1, 8:10]).any())


def test_rope_on_a_stream_and_in_a_graph():
    import torch
    tq = _tq()
    t = tq.tq_rope_plan()
    q, k, pos = _inputs(50, 8, 2, 5000, 4)
    want_q, want_k = torch.empty_like(q), torch.empty_like(k)
    tq.tq_rope(t, q, k, pos, want_q, want_k)
    side = torch.cuda.Stream()
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tq.tq_rope(t, q, k, pos, qo, ko)
    side.synchronize()
    assert torch.equal(qo, want_q) and torch.equal(ko, want_k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tq.tq_rope(t, q, k, pos, qo, ko)
    q.neg_()
    pos.add_(1)
    g.replay()
    torch.cuda.synchronize()
    tq.tq_rope(t, q, k, pos, want_q, want_k)
    assert torch.equal(qo, want_q) and torch.equal(ko, want_k)
