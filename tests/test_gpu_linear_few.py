"""Products of a few tokens straight from activations, which the product's kernel quantises itself, against their
definition in 64 bits; around the count where the quantisation becomes a launch of its own."""
import numpy as np
import pytest
import torch

from tests import around_ref as R
from tests.test_gpu_linear import check, host, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import w8a8_quantized_moe_b200 as mod
    torch.cuda.set_device(0)
    return mod


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("k", [8, 104, 128, 1000, 4104, 16384])
@pytest.mark.parametrize("inp,smooth", [("bf16", True), ("bf16", False), ("f32", True), ("f32", False)])
def test_few_tokens(M, T, k, inp, smooth):
    """k off the input tiles, tokens of sizes far apart, zero tokens, output rows that are left alone."""
    n = 300 if k < 10000 else 130
    g = torch.Generator(device="cuda")
    g.manual_seed(T * 5 + k)
    wq, sw, bias, s = make(g, n, k, smooth=smooth)
    code, dt = (M.MOE_BF16, torch.bfloat16) if inp == "bf16" else (M.MOE_F32, torch.float32)
    lin = M.moe_w8a8_linear_prepare_codes(M.make_linear_config(n, k, in_dtype=code, out_dtype=M.MOE_F32), wq, sw, bias, s)
    x = torch.randn(T, k, generator=g, device="cuda")
    for t in range(T):
        x[t] *= 10.0 ** (5 * t - 9)                     # the tokens' scales differ by orders of magnitude
        x[t, (37 * t) % k] *= 20
    if T == 4:
        x[2] = 0.0
    x = x.to(dt)
    ws = torch.empty(M.moe_w8a8_linear_workspace_size(lin, T), dtype=torch.uint8, device="cuda")
    y = torch.full((T + 1, n), 123.0, device="cuda")
    M.moe_w8a8_linear_forward(lin, x, T, y, ws)
    M.moe_w8a8_linear_check_status(lin)
    v = host(x) if s is None else (host(x) * host(s)).astype(np.float32)
    xq, sx = R.quantize_rows(v)
    ref, mag = R.linear(xq, sx, host(wq), host(sw), host(bias))
    check(y[:T], ref, mag, False)
    assert (y[T] == 123.0).all()
    if T == 4:
        assert torch.equal(y[2], bias)
    # each token alone, and through strides that keep or leave the 16-byte boundaries: the same bits
    for pad in (8, 3):
        wide = torch.zeros(T, k + pad, dtype=dt, device="cuda")[:, :k]
        wide.copy_(x)
        z = torch.empty(T, n, device="cuda")
        M.moe_w8a8_linear_forward(lin, wide, T, z, ws)
        assert torch.equal(z, y[:T])
    for t in range(T):
        z = torch.empty(1, n, device="cuda")
        M.moe_w8a8_linear_forward(lin, x[t:t + 1], 1, z, ws)
        assert torch.equal(z[0], y[t])


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("k", [104, 1000, 4096])
@pytest.mark.parametrize("inp", ["bf16", "f32"])
def test_few_tokens_that_are_not_finite(M, T, k, inp):
    """A token that holds an infinity or a NaN anywhere gets NaN; the others are as without it."""
    n = 150
    g = torch.Generator(device="cuda")
    g.manual_seed(T + k)
    wq, sw, bias, s = make(g, n, k)
    code, dt = (M.MOE_BF16, torch.bfloat16) if inp == "bf16" else (M.MOE_F32, torch.float32)
    lin = M.moe_w8a8_linear_prepare_codes(M.make_linear_config(n, k, in_dtype=code, out_dtype=M.MOE_F32), wq, sw, bias, s)
    x = torch.randn(T, k, generator=g, device="cuda").to(dt)
    ws = torch.empty(M.moe_w8a8_linear_workspace_size(lin, T), dtype=torch.uint8, device="cuda")
    y0, y1 = torch.empty(T, n, device="cuda"), torch.empty(T, n, device="cuda")
    M.moe_w8a8_linear_forward(lin, x, T, y0, ws)
    assert torch.isfinite(y0).all()
    for bad in range(T):
        for at, v in ((0, float("nan")), (k - 1, float("inf")), (k // 2, -float("inf"))):
            z = x.clone()
            z[bad, at] = v
            M.moe_w8a8_linear_forward(lin, z, T, y1, ws)
            for t in range(T):
                assert torch.isnan(y1[t]).all() if t == bad else torch.equal(y0[t], y1[t])
