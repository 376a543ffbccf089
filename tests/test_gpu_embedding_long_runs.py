"""The embedding's gradient where one token fills many places (padding with a
token of the vocabulary): errors that do not grow with their number.

Bound: a chunk's sum goes through at most 64 additions in fp32; the chunks'
sums are added up in 64 bits and rounded once, the scale's product and the
addition to an existing gradient once each."""
import pytest
import torch

import orthogonalizing_optimizer_amd as d3
from tests.layer_ref import EPS32, close, d

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("T,m,dtype", [(1 << 20, 5, F32), ((1 << 20) + 17, 8, BF), (8192, 300, F32),
                                       (300000, 2, F32), (1 << 22, 4, BF)])
def test_one_token_everywhere(T, m, dtype, accumulate):
    # equal rows: each addition to a long chain is rounded the same way
    row = (torch.arange(1, m + 1, dtype=torch.float32) / 3).to(dtype)
    tokens = torch.full((T,), 3)
    tokens[T // 3] = 1
    tokens[T // 5] = -1
    dw = torch.full((6, m), 0.7, device="cuda")
    out = d3.embedding_grad(tokens.cuda(), row.cuda().repeat(T, 1), 6, 1.5, out=dw, accumulate=accumulate)
    want = torch.zeros(6, m, dtype=torch.float64)
    want[3], want[1] = 1.5 * (T - 2) * d(row), 1.5 * d(row)
    if accumulate:
        want += d(torch.tensor(0.7))
    close(out, want, want.abs() * (64 + 3) * EPS32, (T, m, dtype, accumulate))


def test_random_rows_of_one_token():
    T, m = 1 << 20, 6
    g = torch.Generator().manual_seed(1)
    dy = torch.rand(T, m, generator=g) + 0.5
    dw = d3.embedding_grad(torch.zeros(T, dtype=torch.int32).cuda(), dy.cuda(), 2)
    want = torch.stack([d(dy).sum(0), torch.zeros(m, dtype=torch.float64)])
    close(dw, want, want * (64 + 2) * EPS32)
