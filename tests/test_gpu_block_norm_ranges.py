"""The norms around a block at the ends of their ranges: the largest values, long rows in large batches, rows of zeros
and rows that hold an infinity or a NaN, in the kernel for few rows and in the one for many."""
import numpy as np
import pytest
import torch

from tests import around_ref as R
from tests.test_gpu_block_norm import DT, RMS_U, U32, UBF, host, run_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import w8a8_quantized_moe_b200 as mod
    torch.cuda.set_device(0)
    return mod


@pytest.mark.parametrize("T", [3, 250])
@pytest.mark.parametrize("d", [16384, 16383, 4096])
@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("post", [False, True])
def test_the_largest_values(M, T, d, typ, post):
    """Rows whose values are all of the largest size that the norms take, of either sign."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T + d)
    code = M.MOE_F32 if typ == "f32" else M.MOE_BF16
    largest = torch.tensor(1e17).to(DT[typ])
    if largest.double() > 1e17:
        largest = torch.nextafter(largest, torch.zeros_like(largest))
    sign = lambda: torch.randint(0, 2, (T, d), generator=g, device="cuda") * 2.0 - 1  # noqa: E731
    x = (sign() * largest.cuda()).to(DT[typ])
    b = (sign() * largest.cuda()).to(DT[typ])
    w_post = torch.rand(d, generator=g, device="cuda") + 0.5
    w_pre = torch.rand(d, generator=g, device="cuda") + 0.5
    x_out, n_out = torch.empty_like(x), torch.empty(T, d, device="cuda")
    xq, sx = torch.empty(T, 16384, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    # r = x / 2 + 10 norm(b), or x / 2 + b / 2: within the range too
    cfg = M.make_norm_config(d, code, code, M.MOE_F32, residual_scale=0.5, branch_scale=10.0 if post else 0.5)
    M.moe_w8a8_block_norm(cfg, T, b=b, x=x, w_post=w_post if post else None, w_pre=w_pre, x_out=x_out, n_out=n_out, xq=xq, sx=sx)
    eps = np.float64(np.float32(1e-6))
    p = host(b) / R.rms(host(b), eps) * host(w_post) * 10 if post else 0.5 * host(b)
    r = 0.5 * host(x) + p
    got = host(x_out)
    tol = 1.01 * 32 * U32 * (0.5 * np.abs(host(x)) + np.abs(p)) + 1.01 * (UBF if typ == "bf16" else U32) * np.abs(r)
    assert (np.abs(got - r) <= tol).all()
    inv = 1.0 / R.rms(got, eps)
    n = got * inv * host(w_pre)
    assert (np.abs(host(n_out) - n) <= 1.01 * (RMS_U + 4 * U32) * np.abs(n)).all() and (n != 0).any()
    q, s = R.quantize_rows(got.astype(np.float32) * host(w_pre).astype(np.float32))
    assert np.array_equal(xq[:, :d].cpu().numpy(), q)
    want = s.astype(np.float64) * inv[:, 0]
    assert (want > 0).all() and (np.abs(host(sx) - want) <= 1.01 * (RMS_U + U32) * want).all()
    if post:   # the norm after the block alone: its values are of order one, the input's of order 1e17
        M.moe_w8a8_block_norm(M.make_norm_config(d, code, code, M.MOE_F32), T, b=b, w_post=w_post, x_out=x_out)
        p = host(b) / R.rms(host(b), eps) * host(w_post)
        assert (np.abs(host(x_out) - p) <= 1.01 * (RMS_U + 3 * U32 + (UBF if typ == "bf16" else U32)) * np.abs(p)).all()


@pytest.mark.parametrize("T", [3, 250])
@pytest.mark.parametrize("d", [520, 516, 518, 1001, 4104])
@pytest.mark.parametrize("where", ["channel", "element", "w_post"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_what_stands_at_a_rows_end(M, T, d, where, value):
    """An infinite gate or weight of the row's last channel reaches that channel and, through the rms, the others as the
    formulas have it: the stream is as it is elsewhere, n is finite / infinity = 0 there."""
    b, x = torch.ones(T, d, device="cuda"), torch.full((T, d), 2.0, device="cuda")
    w = torch.ones(d, device="cuda")
    special = torch.ones(d, device="cuda")
    special[-1] = value
    x_out, n_out = torch.empty_like(x), torch.empty_like(x)
    xq, sx = torch.full((T, (d + 15) // 16 * 16), 5, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    gate = {"channel": special, "element": special.expand(T, d).contiguous(), "w_post": None}[where]
    cfg = M.make_norm_config(d, M.MOE_F32, M.MOE_F32, M.MOE_F32, eps=1e-6,
                             gate=M.MOE_GATE_NONE if gate is None else getattr(M, "MOE_GATE_" + where.upper()))
    M.moe_w8a8_block_norm(cfg, T, b=b, x=x, gate=gate, w_post=special if gate is None else w, w_pre=w, x_out=x_out, n_out=n_out,
                          xq=xq, sx=sx)
    # 2 + 1 / sqrt(1 + 1e-6); the sum's, root's and products' roundings
    assert ((x_out[:, :-1].double() - (2 + 1 / np.sqrt(1 + 1e-6))).abs() <= 3 * 20 * U32).all()
    if np.isinf(value):
        assert torch.isinf(x_out[:, -1]).all() and (n_out[:, :-1] == 0).all() and torch.isnan(n_out[:, -1]).all()
    else:
        assert torch.isnan(x_out[:, -1]).all() and torch.isnan(n_out).all()
    assert torch.isnan(sx).all() and (xq[:, :d] == 0).all()


@pytest.mark.parametrize("T", [199, 200, 300])
@pytest.mark.parametrize("d", [4104, 8192, 8200, 16384])
def test_long_rows_in_large_batches(M, T, d):
    """The widest blocks of the kernel for many rows, with and without codes, w_post and a gate, in both types."""
    run_case(M, T, d, "bf16", "bf16", "bf16", False, "none", False, False, False)
    run_case(M, T, d, "bf16", "bf16", "bf16", True, "channel", False, True, True, offset=1.0, inplace=True)
    run_case(M, T, d, "f32", "f32", "f32", True, "element", True, True, False, pad=8)
    run_case(M, T, d, "f32", "f32", "bf16", False, "token", False, True, True)


@pytest.mark.parametrize("T", [7, 250])
@pytest.mark.parametrize("d", [512, 4096, 8192, 16384, 516, 1001])
@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("branch", [False, True])
def test_rows_of_zeros_infinities_and_nan(M, T, d, typ, branch):
    """Zero rows give zeros; a row that holds an infinity or a NaN, in the stream or in the branch, gets codes 0 and the
    scale NaN, and its neighbours are as without it."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T + d)
    code = M.MOE_F32 if typ == "f32" else M.MOE_BF16
    x = torch.randn(T, d, generator=g, device="cuda").to(DT[typ])
    b = torch.randn(T, d, generator=g, device="cuda").to(DT[typ])
    w, w_post = (torch.rand(d, generator=g, device="cuda") + 0.5 for _ in range(2))
    cfg = M.make_norm_config(d, code, code, M.MOE_F32)

    def call():
        x_out, n_out = torch.empty_like(x), torch.empty(T, d, device="cuda")
        xq, sx = torch.full((T, 16384), 5, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        M.moe_w8a8_block_norm(cfg, T, b=b if branch else None, x=x, w_post=w_post if branch else None, w_pre=w, x_out=x_out,
                              n_out=n_out, xq=xq, sx=sx)
        return x_out, n_out, xq[:, :d], sx

    clean = call()
    x[1], b[1] = 0.0, 0.0
    special = {2: float("inf"), 3: float("nan"), 4: -float("inf")}
    for t, v in special.items():
        x[t, (t * 97) % d] = v
    if branch:
        b[5, d - 1] = float("nan")
        b[6, 0] = float("inf")
        special.update({5: 0.0, 6: 0.0})
    x_out, n_out, xq, sx = call()
    for t in range(T):
        if t == 1:
            assert (x_out[t] == 0).all() and (n_out[t] == 0).all() and (xq[t] == 0).all() and sx[t] == 0
        elif t in special:
            assert (xq[t] == 0).all() and torch.isnan(sx[t])
        else:
            assert all(torch.equal(a[t], c[t]) for a, c in zip((x_out, n_out, xq, sx), clean))
    # n of a row with an infinity: finite / infinity = 0, infinity / infinity is no number; a NaN takes the whole row
    at = [(t * 97) % d for t in range(5)]
    for t in (2, 4):
        others = torch.arange(d, device="cuda") != at[t]
        assert torch.isnan(n_out[t, at[t]]) and (n_out[t][others] == 0).all() and torch.isinf(x_out[t, at[t]])
    assert torch.isnan(n_out[3]).all()
