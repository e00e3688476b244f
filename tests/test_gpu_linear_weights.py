"""Products whose weights are at the ends of their ranges."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import w8a8_quantized_moe_b200 as mod
    torch.cuda.set_device(0)
    return mod


@pytest.mark.parametrize("smooth", [False, True])
@pytest.mark.parametrize("T", [2, 40, 300])
def test_weights_that_are_not_finite(M, smooth, T):
    """A channel whose weights hold an infinity or a NaN gives NaN.  The other channels are as without it, but for an
    infinity with smoothing, whose input is then smoothed by an infinite factor for all of them."""
    k, n = 300, 200
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    w = torch.randn(k, n, generator=g, device="cuda")
    ax = torch.rand(k, generator=g, device="cuda") + 0.5 if smooth else None
    x = torch.randn(T, k, generator=g, device="cuda")
    w[:, 0] = 50.0                                      # the largest of every input's weights, in a channel that stays

    def forward():
        lin = M.moe_w8a8_linear_prepare(M.make_linear_config(n, k, 0.5, M.MOE_F32, M.MOE_F32), w, None, ax)
        ws = torch.empty(M.moe_w8a8_linear_workspace_size(lin, T), dtype=torch.uint8, device="cuda")
        y = torch.empty(T, n, device="cuda")
        M.moe_w8a8_linear_forward(lin, x, T, y, ws)
        return y

    clean = forward()
    assert torch.isfinite(clean).all()
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    for c, j, v in ((7, 0, float("nan")), (199, 150, float("nan")), (60, 299, float("inf")), (130, 8, -float("inf"))):
        w[j, c] = v
        bad[c] = True
        y = forward()
        everywhere = smooth and abs(v) == float("inf")
        assert torch.isnan(y[:, bad]).all() and torch.equal(torch.isnan(y[:, ~bad]), torch.full_like(y[:, ~bad], everywhere) > 0)
        if everywhere:
            w[j, c] = 1.0
            bad[c] = False
        else:
            assert torch.equal(y[:, ~bad], clean[:, ~bad])


@pytest.mark.parametrize("T", [3, 300])
def test_weights_past_32_bits(M, T):
    """Codes whose offset passes 32 bits: the last channels of 2^20 channels over 4224 inputs (4.4 GB)."""
    n, k = M.MOE_LINEAR_MAX_N, 4224
    assert n * k > 1 << 32
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    wq = torch.empty(n, k, dtype=torch.int8, device="cuda")
    for a in range(0, n, 1 << 17):
        wq[a:a + (1 << 17)].random_(-127, 128, generator=g)
    sw = torch.rand(n, generator=g, device="cuda")
    lin = M.moe_w8a8_linear_prepare_codes(M.make_linear_config(n, k, out_dtype=M.MOE_F32), wq, sw)
    xq = torch.randint(-127, 128, (T, k), generator=g, device="cuda", dtype=torch.int8)
    sx = torch.rand(T, generator=g, device="cuda")
    y = torch.full((T + 1, n), 9.0, device="cuda")
    M.moe_w8a8_linear_forward_codes(lin, xq, sx, T, y)
    M.moe_w8a8_linear_check_status(lin)
    for a in (0, n // 2 - 100, n - 600):
        ref = (xq.double() @ wq[a:a + 600].double().T) * sx.double()[:, None] * sw[a:a + 600].double()
        # the integer's conversion and two products, each rounded once
        assert ((y[:T, a:a + 600].double() - ref).abs() <= 1.01 * 3 * 2.0 ** -24 * ref.abs()).all()
    assert (y[T] == 9.0).all()
    assert torch.equal(M.moe_w8a8_linear_export(lin)["wq"], wq)


@pytest.mark.parametrize("T", [65536 * 16 + 1])
def test_a_million_tokens(M, T):
    n, k = 8, 32
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    wq = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.rand(n, generator=g, device="cuda")
    lin = M.moe_w8a8_linear_prepare_codes(M.make_linear_config(n, k, out_dtype=M.MOE_F32), wq, sw)
    xq = torch.randint(-127, 128, (T, k), generator=g, device="cuda", dtype=torch.int8)
    sx = torch.rand(T, generator=g, device="cuda")
    y = torch.full((T + 1, n), 9.0, device="cuda")
    M.moe_w8a8_linear_forward_codes(lin, xq, sx, T, y)
    M.moe_w8a8_linear_check_status(lin)
    ref = (xq.double() @ wq.double().T) * sx.double()[:, None] * sw.double()
    assert ((y[:T].double() - ref).abs() <= 1.01 * 3 * 2.0 ** -24 * ref.abs()).all() and (y[T] == 9.0).all()
    xs = torch.randn(T, k, generator=g, device="cuda").bfloat16()
    ws = torch.empty(M.moe_w8a8_linear_workspace_size(lin, T), dtype=torch.uint8, device="cuda")
    M.moe_w8a8_linear_forward(lin, xs, T, y, ws)
    amax = xs.float().abs().amax(1, keepdim=True)
    scale = amax / torch.full_like(amax, 127.0)
    ref = (torch.round(xs.float() / scale).double() @ wq.double().T) * scale.double() * sw.double()
    assert ((y[:T].double() - ref).abs() <= 1.01 * 3 * 2.0 ** -24 * ref.abs()).all() and (y[T] == 9.0).all()
