"""Edges of tq_chunk_attention and tq_prompt_attention: what test_gpu_chunk.py and
test_gpu_prompt.py do not reach (bounds: attention64.py)."""
import pytest

from test_gpu_chunk import Case

pytestmark = pytest.mark.gpu

# (queries, query heads of a group) for the three ways of a chunk: up to 32 and up to 128 rows a
# sequence straight over the pages, more of them after a decompression
WAYS = [(1, 4), (8, 4), (30, 4), (150, 4)]


def _tq():
    from kv_cache_vector_02_b200 import tq
    return tq


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
