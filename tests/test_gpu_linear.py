"""Dense products in 8-bit integers against their definition in 64 bits."""
import numpy as np
import pytest
import torch

from tests import around_ref as R

pytestmark = pytest.mark.gpu
U32, UBF = 2.0 ** -24, 2.0 ** -8   # half a step, relative to the value


@pytest.fixture(scope="module")
def M():
    import w8a8_quantized_moe_b200 as mod
    torch.cuda.set_device(0)
    return mod


def check(y, ref, mag, bf16):
    """One rounding for the integer's conversion and one per product (3 of |acc sx sw|), one for the sum, one for a
    bf16 output; a hundredth more for products of roundings."""
    tol = 1.01 * (3 * U32 * mag + U32 * np.abs(ref)) + (UBF * 1.01 * np.abs(ref) if bf16 else 0.0) + 1e-37
    err = np.abs(y.float().cpu().numpy().astype(np.float64) - ref)
    assert (err <= tol).all(), float((err / tol).max())


def make(g, n, k, bias=True, smooth=True):
    wq = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.rand(n, generator=g, device="cuda") * 0.01
    b = torch.randn(n, generator=g, device="cuda") if bias else None
    s = torch.rand(k, generator=g, device="cuda") + 0.5 if smooth else None
    return wq, sw, b, s


def host(t):
    return None if t is None else t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


SHAPES = [(1, 128, 128), (1, 4096, 4096), (2, 1, 1), (3, 17, 5), (5, 1000, 1111), (16, 130, 257), (17, 4096, 384), (32, 640, 6144),
          (33, 100, 1000), (48, 16384, 130), (64, 2048, 512), (65, 96, 300), (100, 4100, 260), (129, 256, 128),
          (257, 1000, 1111), (300, 512, 20000), (512, 384, 8192), (1000, 1040, 4000), (2049, 200, 2500)]


@pytest.mark.parametrize("T,k,n", SHAPES)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_codes(M, T, k, n, out):
    g = torch.Generator(device="cuda")
    g.manual_seed(T * 7 + k + n)
    wq, sw, b, _ = make(g, n, k, bias=T % 2 == 1)
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    lin = M.moe_w8a8_linear_prepare_codes(
        M.make_linear_config(n, k, out_dtype=M.MOE_BF16 if out == "bf16" else M.MOE_F32), wq, sw, b)
    xq = torch.full((T, (k + 15) // 16 * 16), 77, dtype=torch.int8, device="cuda")   # what follows a row's codes is not used
    xq[:, :k] = torch.randint(-128, 128, (T, k), generator=g, device="cuda", dtype=torch.int8)
    sx = torch.rand(T, generator=g, device="cuda")
    y = torch.full((T + 1, n), 123.0, dtype=dt, device="cuda")
    M.moe_w8a8_linear_forward_codes(lin, xq, sx, T, y)
    M.moe_w8a8_linear_check_status(lin)
    ref, mag = R.linear(host(xq)[:, :k], host(sx), host(wq), host(sw), host(b))
    check(y[:T], ref, mag, out == "bf16")
    assert (y[T] == 123.0).all()
    got = M.moe_w8a8_linear_export(lin)
    assert torch.equal(got["wq"], wq) and torch.equal(got["sw"], sw) and got["inv_s"] is None


@pytest.mark.parametrize("T,k,n", [(1, 4096, 256), (7, 100, 33), (64, 1001, 129), (200, 2048, 500), (700, 256, 3000)])
@pytest.mark.parametrize("inp,out,smooth", [("bf16", "bf16", True), ("f32", "f32", False), ("bf16", "f32", True)])
def test_forward(M, T, k, n, inp, out, smooth):
    g = torch.Generator(device="cuda")
    g.manual_seed(T + k + n)
    wq, sw, b, s = make(g, n, k, smooth=smooth)
    code = {"f32": M.MOE_F32, "bf16": M.MOE_BF16}
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}
    lin = M.moe_w8a8_linear_prepare_codes(M.make_linear_config(n, k, in_dtype=code[inp], out_dtype=code[out]), wq, sw, b, s)
    x = torch.randn(T, k, generator=g, device="cuda")
    x[:, 0] *= 30
    if T > 2:
        x[1] = 0.0
        x[2] *= 1e-30
    x = x.to(dt[inp])
    y = torch.empty(T, n, dtype=dt[out], device="cuda")
    ws = torch.empty(M.moe_w8a8_linear_workspace_size(lin, T), dtype=torch.uint8, device="cuda")
    M.moe_w8a8_linear_forward(lin, x, T, y, ws)
    v = host(x) if s is None else (host(x) * host(s)).astype(np.float32)
    xq, sx = R.quantize_rows(v)
    ref, mag = R.linear(xq, sx, host(wq), host(sw), host(b))
    check(y, ref, mag, out == "bf16")
    # the same call again gives the same bits
    y2 = torch.empty_like(y)
    M.moe_w8a8_linear_forward(lin, x, T, y2, ws)
    assert torch.equal(y, y2)
    # strided rows, off the 16-byte boundaries, of x and y; what lies between them stays
    xs = torch.zeros(T, k + 3, dtype=x.dtype, device="cuda")[:, 1:k + 1]
    xs.copy_(x)
    yb = torch.full((T, n + 5), 9.0, dtype=y.dtype, device="cuda")
    M.moe_w8a8_linear_forward(lin, xs, T, yb[:, 2:n + 2], ws)
    assert torch.equal(yb[:, 2:n + 2], y) and (yb[:, :2] == 9).all() and (yb[:, n + 2:] == 9).all()


def test_prepare_from_weights(M):
    """Smoothing and per-channel codes as for the experts: s = ax^a / aw^(1 - a), codes of fp32(s w)."""
    k, n, alpha = 300, 77, 0.6
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    w = torch.randn(k, n, generator=g, device="cuda") * 0.05
    w[:, 5] = 0.0
    ax = torch.rand(k, generator=g, device="cuda") * 10
    ax[4] = 0.0
    bias = torch.randn(n, generator=g, device="cuda")
    for absmax in (ax, None):
        lin = M.moe_w8a8_linear_prepare(M.make_linear_config(n, k, alpha, M.MOE_F32, M.MOE_F32), w, bias, absmax)
        got = M.moe_w8a8_linear_export(lin)
        wh = host(w)
        if absmax is not None:
            a, aw = np.maximum(host(ax).astype(np.float64), np.float32(1e-5)), np.abs(wh).max(1).astype(np.float64)
            s = (a ** np.float64(np.float32(alpha)) / aw ** (1 - np.float64(np.float32(alpha)))).astype(np.float32)
            inv = (1.0 / s.astype(np.float64)).astype(np.float32)
            assert np.allclose(host(got["inv_s"]), inv, rtol=2 * U32, atol=0)
            # the library's own s, for the codes: one rounding of pow may differ
            sl = (1.0 / host(got["inv_s"]).astype(np.float64))
            assert np.allclose(sl, s, rtol=4 * U32)
            q, sc = R.quantize_rows((wh * s[:, None]).astype(np.float32).T.copy())
        else:
            assert got["inv_s"] is None
            q, sc = R.quantize_rows(wh.T.copy())
            assert np.array_equal(host(got["wq"]), q) and np.array_equal(host(got["sw"]), sc)
        assert np.abs(host(got["wq"]).astype(int) - q).max() <= 1 and np.allclose(host(got["sw"]), sc, rtol=4 * U32)
        x = torch.randn(9, k, generator=g, device="cuda")
        y = torch.empty(9, n, device="cuda")
        ws = torch.empty(M.moe_w8a8_linear_workspace_size(lin, 9), dtype=torch.uint8, device="cuda")
        M.moe_w8a8_linear_forward(lin, x, 9, y, ws)
        v = host(x) if absmax is None else (host(x) * host(got["inv_s"])).astype(np.float32)
        xq, sx = R.quantize_rows(v)
        ref, mag = R.linear(xq, sx, host(got["wq"]), host(got["sw"]), host(bias))
        check(y, ref, mag, False)


def test_non_finite_tokens(M):
    """A token that holds an infinity or a NaN gets NaN; its neighbours are as without it."""
    k, n, T = 200, 150, 6
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    wq, sw, b, s = make(g, n, k)
    lin = M.moe_w8a8_linear_prepare_codes(M.make_linear_config(n, k, 0.6, M.MOE_F32, M.MOE_F32), wq, sw, b, s)
    x = torch.randn(T, k, generator=g, device="cuda")
    ws = torch.empty(M.moe_w8a8_linear_workspace_size(lin, T), dtype=torch.uint8, device="cuda")
    y0, y1 = torch.empty(T, n, device="cuda"), torch.empty(T, n, device="cuda")
    M.moe_w8a8_linear_forward(lin, x, T, y0, ws)
    x[1, 7], x[3, 199], x[4, 0] = float("inf"), float("nan"), -float("inf")
    M.moe_w8a8_linear_forward(lin, x, T, y1, ws)
    for t in range(T):
        assert torch.isnan(y1[t]).all() if t in (1, 3, 4) else torch.equal(y0[t], y1[t])


def test_streams_and_graph(M):
    """A call on another stream, and one captured into a graph and replayed with other inputs."""
    T, k, n = 40, 512, 700
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    wq, sw, b, s = make(g, n, k)
    lin = M.moe_w8a8_linear_prepare_codes(M.make_linear_config(n, k), wq, sw, b, s)
    xs = [torch.randn(T, k, generator=g, device="cuda").bfloat16() for _ in range(2)]
    size = M.moe_w8a8_linear_workspace_size(lin, T)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    want = []
    for x in xs:
        y = torch.empty(T, n, dtype=torch.bfloat16, device="cuda")
        M.moe_w8a8_linear_forward(lin, x, T, y, ws)
        want.append(y)
    torch.cuda.synchronize()
    st, y, wsb = torch.cuda.Stream(), torch.empty_like(want[0]), torch.empty_like(ws)
    M.moe_w8a8_linear_forward(lin, xs[1], T, y, wsb, stream=st)
    st.synchronize()
    assert torch.equal(y, want[1])
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.moe_w8a8_linear_forward(lin, x, T, y, wsb)
    for i in (1, 0, 1):
        x.copy_(xs[i])
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
