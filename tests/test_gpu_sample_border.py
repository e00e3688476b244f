"""Sampling where the top_p cut and the order of a list's tokens are decided closely."""
import numpy as np
import pytest
import torch

from tests.test_gpu_sample import check, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import w8a8_quantized_moe_b200 as mod
    torch.cuda.set_device(0)
    return mod


@pytest.mark.parametrize("n", [1, 2, 3, 31, 33, 127, 128, 129, 200, 256, 257, 511, 512, 513, 1000, 2047, 2048, 2049, 3000])
@pytest.mark.parametrize("vocab", [4000, 50000])
def test_lists_of_every_length(M, n, vocab):
    """Lists ordered by counting (up to 128 tokens), by sorting (512), by bins (2048) and longer ones, by top_k and by
    top_p, with equal logits among them."""
    rng = np.random.default_rng(n + vocab)
    rows = 6
    x = np.full((rows, vocab), -60.0, np.float32)
    for r in range(rows):
        at = rng.choice(vocab, n, replace=False)
        x[r, at] = rng.integers(0, 40, n) / np.float32(16) if r % 2 else rng.uniform(0, 3, n)
    u = rng.random(rows).astype(np.float32)
    u[0], u[1] = 0.0, 1 - 2.0 ** -24
    p = rng.uniform(0.3, 0.98, rows).astype(np.float32)
    check(M, dev(x), u, top_k=np.full(rows, n, np.int32))
    check(M, dev(x), u, top_k=rng.integers(1, n + 1, rows).astype(np.int32), top_p=p)
    check(M, dev(x), u, top_p=p)
    check(M, dev(x), u, top_p=p, min_p=rng.uniform(0.05, 0.6, rows).astype(np.float32))
