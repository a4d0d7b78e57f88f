"""The embedding and its gradient against 64 bits (tests/model_refs.py derives
the bounds)."""

import pytest
import torch

import ring_allreduce_rs_amd as ar
from tests import model_refs as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32
I32, I64 = torch.int32, torch.int64


def words(shape, vocab, seed, dtype=I64, pad=0.1):
    """Ids as a text has them: a few of them often; some outside the vocabulary."""
    g = torch.Generator().manual_seed(seed)
    ids = (torch.rand(shape, generator=g, dtype=torch.float64) * torch.log(torch.tensor(vocab + 1.0))
           ).exp().sub(1).long().clamp(0, vocab - 1)
    gone = torch.rand(shape, generator=g)
    ids[gone < pad / 2] = -1
    ids[gone > 1 - pad / 2] = vocab
    return ids.to(dtype).cuda()


def check(ids, vocab, hidden, t, scale, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    table = torch.randn((vocab, hidden), generator=g, device="cuda").to(t)
    y, tol = ref.embedding(table, ids, scale)
    ref.close(ar.embedding(table, ids, scale), y, tol, "y")
    dy = torch.randn((*ids.shape, hidden), generator=g, device="cuda").to(t)
    d, tol = ref.embedding_backward(dy, ids, vocab, scale)
    got = ar.embedding_backward(dy, ids, vocab, scale)
    ref.close(got, d, tol, "dtable")
    assert torch.equal(got, ar.embedding_backward(dy, ids, vocab, scale))     # to the bit


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("tokens,vocab,hidden", [
    (1, 1, 1), (1, 7, 8), (3, 1000, 64), (4, 2000, 4096), (63, 255, 5), (64, 256, 12), (65, 257, 31),
    (200, 300, 771), (1000, 50, 264), (1025, 5000, 100), (2047, 1023, 1001), (5000, 40000, 72),
    (300, 20, 8200)])
def test_there_and_back(tokens, vocab, hidden, t):
    for dtype, scale in ((I64, 1.0), (I32, 64.0)):
        check(words((tokens,), vocab, tokens, dtype), vocab, hidden, t, scale, tokens)


@pytest.mark.parametrize("tokens", [64, 65, 128, 129, 1000, 32768, 32769, 70001])
def test_one_token_takes_all_or_none(tokens):
    for value in (0, 5, 699, -1, 700, 2 ** 40 + 3, -2 ** 62):
        ids = torch.full((tokens,), value, dtype=I64, device="cuda")
        check(ids, 700, 12, F32, -0.5)


@pytest.mark.parametrize("tokens,vocab", [(32768, 3000), (32769, 3000), (40000, 1), (50000, 257),
                                          (100003, 300000), (200000, 1025), (33000, 1 << 20)])
@pytest.mark.parametrize("dtype", [I32, I64])
def test_many_tokens(tokens, vocab, dtype):
    """More tokens than a block of the sort walks by itself."""
    check(words((tokens,), vocab, 5, dtype), vocab, 16, BF, 1.0)


def test_runs_that_meet_in_a_piece():
    """Ids that come 1 .. 200 times, so that their runs begin and end everywhere."""
    ids = torch.cat([torch.full((n,), n) for n in range(200, 0, -1)]).cuda()
    ids = ids[torch.randperm(ids.numel(), generator=torch.Generator().manual_seed(1)).cuda()]
    for t in (BF, F32):
        check(ids, 201, 40, t, 2.0)


def test_shapes_strides_and_none():
    check(words((3, 5, 7), 90, 2), 90, 33, BF, 3.0)
    check(torch.tensor(4, device="cuda"), 9, 16, F32, 1.0)
    d = ar.embedding_backward(torch.empty((0, 24), device="cuda"),
                              torch.empty(0, dtype=I64, device="cuda"), 70, 1.0)
    assert d.shape == (70, 24) and not d.any()
    assert ar.embedding(torch.ones((5, 3), device="cuda"),
                        torch.empty((2, 0), dtype=I32, device="cuda")).shape == (2, 0, 3)
    ids = words((50,), 20, 3)
    base = torch.randn(50 * 40 + 64, device="cuda")
    for off, width in ((0, 32), (1, 33), (3, 7)):
        dy = base[off:off + 50 * 40].view(50, 40)[:, :width]
        d, tol = ref.embedding_backward(dy, ids, 20, 1.0)
        ref.close(ar.embedding_backward(dy, ids, 20), d, tol)


def test_infinities_stay_in_their_rows():
    ids = torch.tensor([1, 2, 1, 3], device="cuda")
    dy = torch.ones((4, 19), device="cuda")
    dy[0, 4], dy[2, 5], dy[3, 18] = torch.inf, torch.nan, -torch.inf
    d, tol = ref.embedding_backward(dy, ids, 5, 2.0)
    ref.close(ar.embedding_backward(dy, ids, 5, 2.0), d, tol)
