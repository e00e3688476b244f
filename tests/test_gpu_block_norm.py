"""The norms around a block against their definition in 64 bits."""
import numpy as np
import pytest
import torch

from tests import around_ref as R

pytestmark = pytest.mark.gpu
U32, UBF = 2.0 ** -24, 2.0 ** -8
# A row's sum of squares: at most 16 sums in a thread, 5 + 5 over the threads, the square itself, and the mean's and
# eps's roundings: 29 half steps relative to a sum of positive terms; half of that through the root, and the root's own
# rounding: 16.
RMS_U = 16 * U32


@pytest.fixture(scope="module")
def M():
    import w8a8_quantized_moe_b200 as mod
    torch.cuda.set_device(0)
    return mod


def host(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def run_case(M, T, d, inp, res, out, post, gate, sigmoid, codes, smooth, offset=0.0, scales=(0.9, 1.25), pad=0, seed=0,
             inplace=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + T * 31 + d)
    code = {"f32": M.MOE_F32, "bf16": M.MOE_BF16}

    def mat(dt, scale=1.0):
        base = torch.full((T, d + pad), 55.0, dtype=dt, device="cuda")
        base[:, :d] = (torch.randn(T, d, generator=g, device="cuda") * scale).to(dt)
        return base[:, :d]

    vec = lambda: torch.rand(d, generator=g, device="cuda") + 0.5  # noqa: E731
    b, x = mat(DT[inp], 2.0), mat(DT[res], 3.0)
    w_post, w_pre, inv_s = vec() if post else None, vec(), vec() if smooth else None
    gt = {"none": None, "token": torch.randn(T, generator=g, device="cuda"), "channel": torch.randn(d, generator=g, device="cuda"),
          "element": mat(DT[inp])}[gate]
    cfg = M.make_norm_config(d, code[inp], code[res], code[out], getattr(M, "MOE_GATE_" + gate.upper()), sigmoid, 1e-5, *scales,
                             weight_offset=offset)
    x0, b0 = host(x), host(b)
    x_out = x if inplace else mat(DT[res])
    n_out = b if inplace and inp == out else mat(DT[out])
    ldq = (d + 15) // 16 * 16 + (16 if pad else 0)
    xq = torch.full((T + 1, ldq), 99, dtype=torch.int8, device="cuda") if codes else None
    sx = torch.full((T + 1,), 7.0, device="cuda") if codes else None
    M.moe_w8a8_block_norm(cfg, T, b=b, x=x, gate=gt, w_post=w_post, w_pre=w_pre, inv_s=inv_s if codes else None, x_out=x_out,
                          n_out=n_out, xq=xq, sx=sx)
    torch.cuda.synchronize()
    # r: the norm (16 + 2 half steps), the gate (sigmoid: 2 units of exp, the sum, the quotient: 6), three products and the sum
    off = np.float64(np.float32(offset))
    p = b0
    if post:
        p = p / R.rms(p, np.float64(np.float32(1e-5))) * (host(w_post) + off)
    if gt is not None:
        gv = host(gt)
        gv = 1.0 / (1.0 + np.exp(-gv)) if sigmoid else gv
        p = p * (gv[:, None] if gate == "token" else gv)
    a, c = (np.float64(np.float32(v)) for v in scales)
    r = a * x0 + c * p
    tol = 1.01 * 32 * U32 * (np.abs(a * x0) + np.abs(c * p)) + 1.01 * (UBF if res == "bf16" else U32) * np.abs(r) + 1e-37
    got = host(x_out)
    assert (np.abs(got - r) <= tol).all(), float((np.abs(got - r) / tol).max())
    # n and the codes are held to the r that was kept
    inv = 1.0 / R.rms(got, np.float64(np.float32(1e-5)))
    n = got * inv * (host(w_pre) + off)
    tol = 1.01 * (RMS_U + 3 * U32 + (UBF if out == "bf16" else U32)) * np.abs(n) + 1e-37
    assert (np.abs(host(n_out) - n) <= tol).all(), float((np.abs(host(n_out) - n) / tol).max())
    if codes:
        v = got.astype(np.float32) * (host(w_pre).astype(np.float32) + np.float32(offset))
        v = v if inv_s is None else v * host(inv_s).astype(np.float32)
        q, s = R.quantize_rows(v)
        assert np.array_equal(xq[:T, :d].cpu().numpy(), q)
        want = s.astype(np.float64) * inv[:, 0]
        assert (np.abs(host(sx)[:T] - want) <= 1.01 * (RMS_U + U32) * want + 1e-37).all()
        assert (xq[:T, d:] == 99).all() and (xq[T] == 99).all() and sx[T] == 7.0
    for t in (x_out, n_out):
        whole = t._base if t._base is not None else t
        assert (whole[:, d:] == 55).all()


@pytest.mark.parametrize("d", [1, 8, 33, 64, 128, 256, 257, 512, 513, 1000, 1001, 1024, 1032, 2048, 2056, 4096, 4097, 4104, 5000,
                               8192, 8200, 9999, 16383, 16384])
@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_sizes(M, d, typ):
    run_case(M, 9, d, typ, typ, typ, True, "channel", False, True, True)
    run_case(M, 1, d, typ, typ, typ, False, "none", False, True, False)


@pytest.mark.parametrize("gate", ["none", "token", "channel", "element"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("post", [False, True])
def test_gates(M, gate, sigmoid, post):
    for d, pad in ((520, 0), (520, 8), (520, 3), (777, 0)):
        run_case(M, 13, d, "bf16", "f32", "bf16", post, gate, sigmoid, True, True, offset=1.0, pad=pad)
        run_case(M, 13, d, "f32", "bf16", "f32", post, gate, sigmoid, False, False, pad=pad)


def test_in_place_and_many_rows(M):
    for d in (64, 1000, 4096):
        run_case(M, 3001, d, "bf16", "bf16", "bf16", True, "token", True, True, True, inplace=True)
        run_case(M, 301, d, "f32", "f32", "f32", False, "none", False, False, False, inplace=True, scales=(1.0, 1.0))


def test_parts(M):
    """Without a branch, without a stream, without a norm: each part that a call may leave out."""
    T, d = 5, 200
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(T, d, generator=g, device="cuda")
    w = torch.rand(d, generator=g, device="cuda") + 0.5
    cfg = M.make_norm_config(d, M.MOE_F32, M.MOE_F32, M.MOE_F32)
    out = [torch.empty(T, d, device="cuda") for _ in range(5)]
    M.moe_w8a8_block_norm(cfg, T, x=x, w_pre=w, n_out=out[0])                       # the norm alone
    M.moe_w8a8_block_norm(cfg, T, b=x, w_pre=w, n_out=out[1], x_out=out[2])         # a branch on no stream
    M.moe_w8a8_block_norm(cfg, T, b=x, w_post=w, x_out=out[3])                      # the norm after a block alone
    assert torch.equal(out[0], out[1]) and torch.equal(out[2], x)
    ref = host(x) / R.rms(host(x), np.float64(np.float32(1e-6))) * host(w)
    for i in (0, 3):
        assert (np.abs(host(out[i]) - ref) <= 1.01 * (RMS_U + 3 * U32) * np.abs(ref) + 1e-37).all()
    xq, sx = torch.empty(T, 208, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    M.moe_w8a8_block_norm(cfg, T, x=x, xq=xq, sx=sx)                                # the quantisation of a token alone
    q, s = R.quantize_rows(x.cpu().numpy())
    assert np.array_equal(xq[:, :d].cpu().numpy(), q) and np.array_equal(sx.cpu().numpy(), s)


def test_zero_and_non_finite_rows(M):
    T, d = 6, 300
    x = torch.ones(T, d, device="cuda")
    x[1] = 0.0
    x[2, 5], x[3, 299], x[4, 0] = float("inf"), float("nan"), -float("inf")
    w = torch.ones(d, device="cuda")
    n = torch.empty(T, d, device="cuda")
    xq, sx = torch.full((T, 304), 5, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    cfg = M.make_norm_config(d, M.MOE_F32, M.MOE_F32, M.MOE_F32)
    M.moe_w8a8_block_norm(cfg, T, x=x, w_pre=w, n_out=n, xq=xq, sx=sx)
    assert (n[1] == 0).all() and sx[1] == 0 and (xq[1:5, :d] == 0).all()
    assert torch.isnan(sx[2:5]).all() and torch.isfinite(sx[[0, 1, 5]]).all()
    assert torch.isnan(n[3, 299]) and (xq[[0, 5], :d] == 127).all()


def test_stream_and_graph(M):
    T, d = 33, 4096
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    b = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    w = torch.rand(d, generator=g, device="cuda")
    cfg = M.make_norm_config(d)
    want = [torch.empty_like(x), torch.empty_like(x)]
    M.moe_w8a8_block_norm(cfg, T, b=b, x=x, w_pre=w, x_out=want[0], n_out=want[1])
    torch.cuda.synchronize()
    got, st = [torch.empty_like(x), torch.empty_like(x)], torch.cuda.Stream()
    M.moe_w8a8_block_norm(cfg, T, b=b, x=x, w_pre=w, x_out=got[0], n_out=got[1], stream=st)
    st.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.moe_w8a8_block_norm(cfg, T, b=b, x=x, w_pre=w, x_out=got[0], n_out=got[1])
    b.neg_(), x.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(-want[0], got[0]) and torch.equal(-want[1], got[1])


@pytest.mark.parametrize("d", [34, 36, 510, 516, 1002, 1004, 2050, 4002, 4004, 5002, 5004, 16380, 16382])
@pytest.mark.parametrize("inp,res,out", [("bf16", "bf16", "bf16"), ("f32", "f32", "f32"), ("bf16", "f32", "bf16")])
def test_rows_on_smaller_boundaries(M, d, inp, res, out):
    """Widths that divide by 2 or 4 only, and strides that do."""
    run_case(M, 7, d, inp, res, out, True, "element", True, True, True)
    run_case(M, 5, d, inp, res, out, False, "none", False, True, False, pad=2)
    run_case(M, 3, d, inp, res, out, True, "token", False, False, False, pad=1)


@pytest.mark.parametrize("T", [1, 7, 8, 9, 199, 200, 201, 2500])
@pytest.mark.parametrize("d", [40, 256, 512, 520, 1024, 2048, 2560, 4096])
def test_row_counts(M, T, d):
    """Both kernels of rows on 16-byte boundaries, at the count where one takes over from the other."""
    run_case(M, T, d, "bf16", "bf16", "bf16", True, "channel", True, True, True, offset=1.0)
    run_case(M, T, d, "f32", "f32", "bf16", False, "none", False, True, True)
    run_case(M, T, d, "bf16", "bf16", "f32", False, "element", False, False, False, pad=8)


@pytest.mark.parametrize("T", [3, 250])
@pytest.mark.parametrize("d", [512, 516, 1001])
@pytest.mark.parametrize("inp,res", [("bf16", "f32"), ("f32", "bf16")])
def test_branch_without_a_stream_of_another_type(M, T, d, inp, res):
    """No x: the new stream still has its own type, which x_out and the norm's input are rounded to."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T + d)
    code = {"f32": M.MOE_F32, "bf16": M.MOE_BF16}
    b = torch.randn(T, d, generator=g, device="cuda").to(DT[inp])
    w = torch.rand(d, generator=g, device="cuda") + 0.5
    x_out = torch.full((T + 1, d), 9.0, dtype=DT[res], device="cuda")
    n_out = torch.full((T + 1, d), 9.0, device="cuda")
    xq, sx = torch.empty(T, (d + 15) // 16 * 16, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    M.moe_w8a8_block_norm(M.make_norm_config(d, code[inp], code[res], M.MOE_F32), T, b=b, w_pre=w, x_out=x_out, n_out=n_out,
                          xq=xq, sx=sx)
    assert torch.equal(x_out[:T], b.float().to(DT[res])) and (x_out[T] == 9).all() and (n_out[T] == 9).all()
    r = host(x_out[:T])
    n = r / R.rms(r, np.float64(np.float32(1e-6))) * host(w)
    assert (np.abs(host(n_out[:T]) - n) <= 1.01 * (RMS_U + 4 * U32) * np.abs(n) + 1e-37).all()
    q, _ = R.quantize_rows(r.astype(np.float32) * host(w).astype(np.float32))
    assert np.array_equal(xq[:, :d].cpu().numpy(), q)
