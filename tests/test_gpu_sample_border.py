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


@pytest.mark.parametrize("vocab", [5000, 40001, 262144])
@pytest.mark.parametrize("temperature", [1.0, 0.7, 3.0])
def test_a_cut_beside_a_far_tail(M, vocab, temperature):
    """Masses 1 and 0.01 at the head and 0.006 in all other tokens together, far below: whether the second token is kept
    turns on the tail's sum, which is held to 2^-23 of the largest mass, beside sums within 3e-9 of theirs; top_p and the
    product with it are rounded to 2^-24 and 2^-53.  So a top_p four fp32 steps (2^-22) or more from the border decides
    as the definition does."""
    rng = np.random.default_rng(vocab)
    t = np.float64(np.float32(temperature))
    x = (t * (np.log(0.006 / vocab) + 0.2 * rng.standard_normal(vocab))).astype(np.float32)
    first, second = vocab // 3, vocab - 2
    x[first], x[second] = 0.0, np.float32(t * np.log(0.01))
    e = np.exp(x.astype(np.float64) / t)
    border = np.float32(1.0 / e.sum())                  # the first token alone reaches up to this top_p
    steps = np.array([-4096, -256, -16, -4, 4, 16, 256, 4096])
    top_p = (border + steps * 2.0 ** -24).astype(np.float32)
    assert (np.abs(top_p.astype(np.float64) * e.sum() - 1.0) >= 3.4 * 2.0 ** -24).all() and (1 - top_p > 0.011).all()
    rows = len(steps)
    logits = dev(np.tile(x, (rows, 1)))
    u = np.full(rows, 1 - 2.0 ** -24, np.float32)       # the last token that is kept
    check(M, logits, u, top_p=top_p, temperature=np.full(rows, temperature, np.float32))
    check(M, logits, u * 0, top_p=top_p, temperature=np.full(rows, temperature, np.float32))


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


def test_settings_that_are_no_numbers(M):
    """A NaN top_p or min_p is off, a NaN u is 0."""
    rng = np.random.default_rng(5)
    f = np.float32
    for vocab in (300, 30000):
        x = rng.standard_normal((4, vocab)).astype(f) * 3
        u = rng.random(4).astype(f)
        nan = np.full(4, np.nan, f)
        check(M, dev(x), u, top_p=nan)
        check(M, dev(x), u, min_p=nan)
        check(M, dev(x), u, top_k=np.full(4, 20, np.int32), top_p=nan, min_p=nan)
        tokens = [torch.empty(4, dtype=torch.int32, device="cuda") for _ in range(2)]
        M.moe_w8a8_sample(dev(x), dev(nan), tokens[0], top_p=dev(np.full(4, 0.8, f)))
        M.moe_w8a8_sample(dev(x), dev(u * 0), tokens[1], top_p=dev(np.full(4, 0.8, f)))
        assert torch.equal(*tokens)


def test_the_most_rows(M):
    rows, vocab = M.MOE_SAMPLE_MAX_ROWS, 33
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(rows, vocab, generator=g, device="cuda")
    u = torch.rand(rows, generator=g, device="cuda")
    token = torch.full((rows + 1,), 99, dtype=torch.int32, device="cuda")
    M.moe_w8a8_sample(x, u, token, temperature=torch.zeros(rows, device="cuda"))
    assert torch.equal(token[:rows], x.argmax(1).int()) and token[rows] == 99
    M.moe_w8a8_sample(x, u * 0, token)
    assert (token[:rows] == 0).all() and token[rows] == 99
    M.moe_w8a8_sample(x, u, token, top_k=torch.ones(rows, dtype=torch.int32, device="cuda"))
    assert torch.equal(token[:rows], x.argmax(1).int())
