"""Devices of the binding's tensors and contexts, on the CPU: nothing here reaches a device."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture()
def tq():
    from kv_cache_vector_02_b200 import tq as m
    return m


@pytest.mark.parametrize("make", ["tq_init_host", "tq_init_ex"])
def test_host_contexts_ask_for_no_device(tq, monkeypatch, make):
    """As in a forked child of a process that used CUDA: asking for the current device raises."""
    def refuse():
        raise RuntimeError("Cannot re-initialize CUDA in forked subprocess")

    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", refuse)
    ctx = tq.tq_init_host(128, 4, 0) if make == "tq_init_host" else tq.tq_init_ex(128, 4, 0, flags=tq.FLAG_HOST_ONLY)
    assert ctx.device is None
    assert tq.tq_chunk_bytes(ctx, tq.KIND_KEY) > 0


def test_tensors_on_the_host_are_refused(tq):
    """The kernels take device pointers only."""
    table = tq.tq_rope_plan()
    q, k = torch.zeros((4, 8, 128), dtype=torch.float16), torch.zeros((4, 2, 128), dtype=torch.float16)
    pos, cu = torch.zeros(4, dtype=torch.int32), torch.tensor([0, 4], dtype=torch.int32)
    ctx = tq.tq_init_host(128, 4, 0)
    ctx.device = 0  # as a context of device 0
    cache = [torch.zeros((2, 2, tq.tq_chunk_bytes(ctx, kind)), dtype=torch.uint8) for kind in (0, 1)]
    bt, lens = torch.zeros((1, 2), dtype=torch.int32), torch.tensor([4], dtype=torch.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for call in (lambda: tq.tq_rope(table, q, k, pos, stream=0),
                 lambda: tq.tq_rope(table, q, None, pos, stream=0),
                 lambda: tq.tq_prompt_attention(ctx, q, k, k, cu, torch.zeros_like(q), stream=0),
                 lambda: tq.tq_chunk_attention(ctx, q, cu, *cache, bt, lens, 32, torch.zeros_like(q), ws, stream=0)):
        with pytest.raises(tq.TQError) as e:
            call()
        assert e.value.status == tq.TQ_ERR_INVALID_ARG and "must be on" in str(e.value)
