"""Rotary tables (host) and the refusals of tq_rope, on the CPU: nothing here reaches a
device."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def tq():
    from kv_cache_vector_02_b200 import tq as m
    return m


def _theta(rot, base, kind, f, L, low, high):
    """Frequencies from the definitions, in float64, one pair at a time."""
    out = []
    for i in range(rot // 2):
        b = base * f ** (rot / (rot - 2)) if kind == 2 else base
        th = b ** (-2.0 * i / rot)
        if kind == 1:
            th /= f
        if kind == 3:
            wave = 2 * math.pi / th
            if wave > L / low:
                th /= f
            elif wave > L / high:
                u = (L / wave - low) / (high - low)
                th = (1 - u) * th / f + u * th
        if kind == 4:
            at = lambda x: rot * math.log(L / (2 * math.pi * x)) / (2 * math.log(base))  # noqa: E731
            a, z = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
            u = min(max((i - a) / max(z - a, 0.001), 0.0), 1.0)
            th = th * (1 - u) + th / f * u
        out.append(th)
    return np.array(out)


@pytest.mark.parametrize("rot,base,kind,f,L,low,high", [
    (128, 10000.0, 0, 1.0, 0, 0, 0), (2, 10000.0, 0, 1.0, 0, 0, 0), (64, 500000.0, 1, 4.0, 0, 0, 0),
    (96, 10000.0, 2, 8.0, 0, 0, 0), (128, 500000.0, 3, 8.0, 8192, 1.0, 4.0), (128, 10000.0, 4, 16.0, 4096, 1.0, 32.0),
    (20, 1.5, 4, 2.5, 1000, 1.0, 32.0), (80, 1e7, 3, 1.0, 2048, 1.0, 4.0)])
def test_frequencies(tq, rot, base, kind, f, L, low, high):
    t = tq.tq_rope_plan(rot, tq.ROPE_HALF, base, kind, f, L, low, high)
    want = _theta(rot, base, kind, f, L, low, high)
    got = np.array([t.turns[i] for i in range(rot // 2)], dtype=np.float64) * 2.0 ** -64 * 2 * math.pi
    assert np.all(np.abs(got - want) <= 4e-14 * want + 2.0 ** -64 * 2 * math.pi)
    assert t.rot_dim == rot and t.layout == tq.ROPE_HALF
    assert abs(t.mscale - (0.1 * math.log(f) + 1 if kind == 4 else 1.0)) <= 2.0 ** -24 * 2
    assert all(t.turns[i] == 0 for i in range(rot // 2, 64))


@pytest.mark.parametrize("kw,status", [
    (dict(rot_dim=0), 1), (dict(rot_dim=3), 1), (dict(rot_dim=130), 1), (dict(base=1.0), 1),
    (dict(base=float("inf")), 1), (dict(base=float("nan")), 1), (dict(scaling=1, factor=0.5), 1),
    (dict(scaling=1, factor=float("nan")), 1), (dict(scaling=2, factor=2.0, rot_dim=2), 1),
    (dict(scaling=3, factor=2.0), 1), (dict(scaling=3, factor=2.0, original_len=64, low=4.0, high=4.0), 1),
    (dict(scaling=4, factor=2.0, original_len=64, low=0.0, high=4.0), 1), (dict(scaling=5), 2), (dict(scaling=-1), 2),
    (dict(layout=2), 2)])
def test_plan_refuses(tq, kw, status):
    with pytest.raises(tq.TQError) as e:
        tq.tq_rope_plan(**kw)
    assert e.value.status == status


def test_plan_refuses_null(tq):
    assert tq._lib.tq_rope_plan(128, 0, 10000.0, 0, 1.0, 0.0, 0.0, 0.0, None) == tq.TQ_ERR_INVALID_ARG


def _raw(tq, table, q=1 << 20, qs=1024, k=1 << 21, ks=256, T=4, Hq=8, Hkv=2, pos=1 << 22, qo=1 << 23, qos=1024,
         ko=1 << 24, kos=256):
    t = ctypes.byref(table) if table is not None else None
    return tq._lib.tq_rope(t, q, qs, k, ks, T, Hq, Hkv, pos, qo, qos, ko, kos, 0, None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(q=None, k=None), dict(Hq=0), dict(Hkv=0), dict(pos=None), dict(qo=None), dict(ko=None),
    dict(qs=1020), dict(qs=1016), dict(kos=248), dict(q=(1 << 20) + 8), dict(ko=(1 << 24) + 2),
    dict(qo=(1 << 20) + 256),               # over its own input, shifted
    dict(qo=1 << 20, qos=2048),             # its own input with another stride
    dict(ko=1 << 20),                       # over the other input
    dict(ko=(1 << 23) + 16),                # over the other output
    dict(qo=(1 << 22) - 16, T=1),           # over the positions
])
def test_rope_refuses(tq, kw):
    assert _raw(tq, tq.tq_rope_plan(), **kw) == tq.TQ_ERR_INVALID_ARG


def test_rope_refuses_tables(tq):
    assert _raw(tq, None) == tq.TQ_ERR_INVALID_ARG
    for field, value in (("rot_dim", 0), ("rot_dim", 130), ("rot_dim", 7), ("layout", 3)):
        t = tq.tq_rope_plan()
        setattr(t, field, value)
        assert _raw(tq, t) == tq.TQ_ERR_INVALID_ARG
    assert _raw(tq, tq.tq_rope_plan(), T=0, pos=None) == tq.TQ_OK


def test_binding_refuses(tq):
    t = tq.tq_rope_plan()
    q, k = torch.zeros((4, 8, 128), dtype=torch.float16), torch.zeros((4, 2, 128), dtype=torch.float16)
    pos = torch.zeros(4, dtype=torch.int32)
    for bad in (dict(q=q.float()), dict(q=q[:, :, :64]), dict(q=q.transpose(0, 1)), dict(k=k[:3]), dict(positions=pos.long()),
                dict(positions=pos[:3]), dict(q_out=q[:, :4]), dict(q=None, q_out=q), dict(q=None, k=None),
                dict(q=q[:1].expand(4, 8, 128))):
        args = dict(q=q, k=k, positions=pos) | bad
        with pytest.raises(tq.TQError) as e:
            tq.tq_rope(t, stream=0, **args)
        assert e.value.status == tq.TQ_ERR_INVALID_ARG
    # nothing to do: no launch
    tq.tq_rope(t, q[:0], k[:0], pos[:0], stream=0)


def test_prompt_binding_refuses(tq):
    ctx = tq.tq_init_host(128, 4, 0)
    q, k = torch.zeros((4, 8, 128), dtype=torch.float16), torch.zeros((4, 2, 128), dtype=torch.float16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    out = torch.zeros((4, 8, 128), dtype=torch.float32)
    for bad in (dict(q=q.to(torch.bfloat16)), dict(k=k[:3]), dict(v=k[:, :1]), dict(cu_seqlens=cu.long()),
                dict(cu_seqlens=cu[:0]), dict(out=out[:, :4]), dict(out=out.double()), dict(q=q.transpose(0, 1))):
        args = dict(q=q, k=k, v=k, cu_seqlens=cu, out=out) | bad
        with pytest.raises(tq.TQError) as e:
            tq.tq_prompt_attention(ctx, stream=0, **args)
        assert e.value.status == tq.TQ_ERR_INVALID_ARG and ("must" in str(e.value))
    with pytest.raises(tq.TQError) as e:  # the shapes pass; the library refuses a host-only context
        tq.tq_prompt_attention(ctx, q, k, k, cu, out, stream=0)
    assert e.value.status == tq.TQ_ERR_INVALID_ARG and "must" not in str(e.value)
