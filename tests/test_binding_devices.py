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
