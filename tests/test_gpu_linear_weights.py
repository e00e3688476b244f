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
