"""Token sampling against its definition in 64 bits: the same tokens, and their probabilities."""
import numpy as np
import pytest
import torch

from tests import around_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import w8a8_quantized_moe_b200 as mod
    torch.cuda.set_device(0)
    return mod


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check(M, logits, u, **kw):
    """logits: a CUDA tensor [rows][vocab], rows possibly strided."""
    rows, vocab = logits.shape
    token = torch.full((rows + 1,), 77, dtype=torch.int32, device="cuda")
    prob = torch.full((rows + 1,), 7.0, device="cuda")
    allowed = kw.pop("allowed", None)
    bits = None if allowed is None else dev(R.pack_bits(allowed))
    M.moe_w8a8_sample(logits, dev(u), token, prob=prob, allowed=bits, **{k: dev(v) for k, v in kw.items()})
    want, p = R.sample(logits.float().cpu().numpy(), u, allowed=allowed, **kw)
    got, q = token.cpu().numpy(), prob.cpu().numpy()
    assert np.array_equal(got[:rows], want), (got[:rows], want)
    # masses are held to 2^-45 of the largest (2^-27 in all over 2^18 tokens) and exp to 1e-11; one fp32 rounding
    assert (np.abs(q[:rows] - p) <= (1.01 * 2.0 ** -24 + 2.0 ** -27) * p + 1e-37).all()
    assert got[rows] == 77 and q[rows] == 7.0
    # once more, without the probabilities
    again = torch.empty_like(token)
    M.moe_w8a8_sample(logits, dev(u), again, allowed=bits, **{k: dev(v) for k, v in kw.items()})
    assert torch.equal(again[:rows], token[:rows])


def settings(rng, rows, k=True, p=True, m=True, t=True):
    f = np.float32
    return {key: v for key, v, on in [
        ("temperature", np.where(rng.random(rows) < 0.15, 0.0, rng.uniform(0.3, 2.0, rows)).astype(f), t),
        ("top_k", np.where(rng.random(rows) < 0.2, 0, rng.integers(1, 300, rows)).astype(np.int32), k),
        ("top_p", np.where(rng.random(rows) < 0.2, 1.0, rng.uniform(0.05, 0.999, rows)).astype(f), p),
        ("min_p", np.where(rng.random(rows) < 0.3, 0.0, rng.uniform(0.0, 0.3, rows)).astype(f), m)] if on}


VOCABS = [1, 2, 31, 32, 33, 100, 1000, 1001, 8192, 8193, 20000, 32000, 65537, 131072, 151936, 262143, 262144]


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_vocabularies(M, vocab, typ):
    rng = np.random.default_rng(vocab)
    rows = 8
    x = rng.standard_normal((rows, vocab)).astype(np.float32) * 2.5
    logits = dev(x).to(torch.bfloat16 if typ == "bf16" else torch.float32)
    u = rng.random(rows).astype(np.float32)
    u[0], u[-1] = 0.0, np.float32(1 - 2.0 ** -24)
    check(M, logits, u)
    check(M, logits, u, **settings(rng, rows))
    check(M, logits, u, **settings(rng, rows, p=False, m=False))
    check(M, logits, u, **settings(rng, rows, k=False, m=False))


@pytest.mark.parametrize("vocab", [50, 1000, 40000])
def test_masks_and_strides(M, vocab):
    rng = np.random.default_rng(vocab + 1)
    rows = 12
    wide = dev(rng.standard_normal((rows, vocab + 7)).astype(np.float32) * 3)
    logits = wide[:, 3:vocab + 3]                       # rows off the 16-byte boundaries
    allowed = rng.random((rows, vocab)) < 0.3
    allowed[1] = False                                  # nothing may be chosen
    allowed[2] = False
    allowed[2, vocab - 1] = True                        # one token
    allowed[3] = True
    # what stands in the place of a token that may not be chosen does not matter
    junk = torch.tensor([float("nan"), float("inf"), -float("inf"), 3.4e38], device="cuda")
    off = dev(~allowed)
    logits[off] = junk[torch.randint(0, 4, (int(off.sum()),), device="cuda")]
    u = rng.random(rows).astype(np.float32)
    check(M, logits, u, allowed=allowed)
    check(M, logits, u, allowed=allowed, **settings(rng, rows))
    check(M, logits.bfloat16().contiguous(), u, allowed=allowed, **settings(rng, rows))


def test_ties(M):
    """Equal logits: the lowest index first, in the top-k and top-p cuts and for the largest."""
    rng = np.random.default_rng(7)
    for vocab in (64, 3000, 70000):
        rows = 10
        x = rng.integers(-2, 3, (rows, vocab)).astype(np.float32)
        x[0] = 1.0                                      # all equal
        x[1] = -0.0
        x[1, ::2] = 0.0                                 # -0 equals +0
        u = rng.random(rows).astype(np.float32)
        k = np.minimum(rng.integers(1, vocab, rows), vocab).astype(np.int32)
        check(M, dev(x), u, top_k=k)
        check(M, dev(x), u, top_p=rng.uniform(0.01, 0.99, rows).astype(np.float32))
        check(M, dev(x), u, top_k=k, top_p=rng.uniform(0.2, 0.99, rows).astype(np.float32))
        check(M, dev(x), u, temperature=np.zeros(rows, np.float32))


def test_values_at_the_ends(M):
    """Masks of the type's lowest value, infinities, NaN, and settings at and past the ends of their ranges."""
    f = np.float32
    low, inf, nan = np.finfo(f).min, np.inf, np.nan
    x = np.full((12, 500), low, f)
    x[0, 77] = 3.0                                      # one token above the lowest value
    x[1, :] = low                                       # all at the lowest value: they share the mass
    x[2, 10:20] = inf                                   # infinities share the mass
    x[3, :] = -inf                                      # nothing may be chosen
    x[4, :] = nan
    x[5, 3], x[5, 400] = nan, 1.0
    x[6] = np.linspace(-30, 30, 500)
    x[7] = np.linspace(-1e30, 1e30, 500)
    x[8] = np.linspace(-1e-30, 1e-30, 500)
    x[9] = 1e-45
    x[10, 499] = -inf
    x[11] = np.linspace(-5, 5, 500)
    rng = np.random.default_rng(3)
    u = rng.random(12).astype(f)
    one = np.ones(12, f)
    check(M, dev(x), u)
    check(M, dev(x), u, temperature=one * f(1e-20))
    check(M, dev(x), u, temperature=one * f(1e30))
    check(M, dev(x), u, temperature=-one)
    check(M, dev(x), u, top_k=np.full(12, 1 << 30, np.int32))
    check(M, dev(x), u, top_k=np.full(12, -5, np.int32))
    check(M, dev(x), u, top_k=np.full(12, 1, np.int32))
    check(M, dev(x), u, top_p=one * 0)
    check(M, dev(x), u, top_p=one * 2)
    check(M, dev(x), u, top_p=one * f(0.5), min_p=one * f(0.2))
    check(M, dev(x), u, min_p=one * 3)
    check(M, dev(x), one * 0)
    check(M, dev(x), one * f(1 - 2.0 ** -24))


def test_temperatures_that_are_no_numbers(M):
    """A NaN is not above the smallest temperature: greedy.  Infinity counts as 3e38."""
    rng = np.random.default_rng(23)
    for V in (1, 700, 40000):
        x = rng.standard_normal((6, V)).astype(np.float32) * 4
        u = rng.random(6).astype(np.float32)
        t = np.array([np.nan, 1.0, np.nan, np.inf, 3.4e38, -np.inf], np.float32)
        check(M, dev(x), u, temperature=t)
        check(M, dev(x), u, temperature=t, top_k=np.full(6, 5, np.int32), top_p=np.full(6, 0.5, np.float32))
        check(M, dev(x), u, temperature=t, min_p=np.full(6, 0.5, np.float32))


def test_many_rows_and_flat_masses(M):
    rng = np.random.default_rng(11)
    x = rng.standard_normal((300, 5000)).astype(np.float32) * 0.5
    check(M, dev(x), rng.random(300).astype(np.float32), **settings(rng, 300))
    x = rng.standard_normal((20, 100000)).astype(np.float32) * 0.3
    check(M, dev(x), rng.random(20).astype(np.float32), top_p=np.full(20, 0.9, np.float32))


def test_stream_and_graph(M):
    rng = np.random.default_rng(12)
    x = dev(rng.standard_normal((16, 30000)).astype(np.float32) * 3)
    u = dev(rng.random(16).astype(np.float32))
    p = torch.full((16,), 0.8, device="cuda")
    want = []
    for sign in (1, -1):
        t = torch.empty(16, dtype=torch.int32, device="cuda")
        M.moe_w8a8_sample(x * sign, u, t, top_p=p)
        want.append(t)
    torch.cuda.synchronize()
    st, got = torch.cuda.Stream(), torch.empty(16, dtype=torch.int32, device="cuda")
    M.moe_w8a8_sample(x, u, got, top_p=p, stream=st)
    st.synchronize()
    assert torch.equal(got, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.moe_w8a8_sample(x, u, got, top_p=p)
    for i in (1, 0):
        x.neg_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want[i])
