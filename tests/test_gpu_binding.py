"""The binding's handling of streams and handles on a GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import w8a8_quantized_moe_b200 as mod
    torch.cuda.set_device(0)
    return mod


def product(M, n=8192, k=4096):
    wq = torch.randint(-127, 128, (n, k), device="cuda", dtype=torch.int8)
    return M.moe_w8a8_linear_prepare_codes(M.make_linear_config(n, k), wq, torch.rand(n, device="cuda")), wq


def layer(M, d=512, f=2048, E=32):
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    return M.moe_w8a8_prepare(M.make_config(d, f, E, 2), r(E, d, f), r(E, d, f), r(E, f, d), r(d, E), r(d).abs())


@pytest.mark.parametrize("what", ["product", "layer"])
@pytest.mark.parametrize("as_int", [False, True])
def test_export_on_another_stream(M, what, as_int):
    """What an export on another stream writes to is no memory that work on the current one still reads."""
    handle, export = (product(M)[0], M.moe_w8a8_linear_export) if what == "product" else (layer(M), M.moe_w8a8_export_weights)
    want = export(handle)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept = torch.empty(40 << 20, dtype=torch.int8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    block = torch.full((40 << 20,), 5, dtype=torch.int8, device="cuda")
    torch.cuda._sleep(200_000_000)                      # about 0.1 s
    kept.copy_(block)
    del block                                           # its memory is free for the current stream's next tensor
    got = export(handle, stream=st.cuda_stream if as_int else st)
    torch.cuda.synchronize()
    assert (kept == 5).all()
    for out in (got, export(handle, stream=0), export(handle, stream=torch.cuda.default_stream())):
        for key, v in want.items():
            assert (v is None and out[key] is None) or torch.equal(v, out[key])


def test_export_after_the_configuration_changed(M):
    """The caller's configuration serves for a second product; the first one's export is whole."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    cfg = M.make_linear_config(300, 500)
    made = []
    for n, k in ((300, 500), (40, 20)):
        cfg.n, cfg.k = n, k
        wq = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
        made.append((M.moe_w8a8_linear_prepare_codes(cfg, wq, torch.rand(n, device="cuda")), wq))
    for lin, wq in made:
        assert torch.equal(M.moe_w8a8_linear_export(lin)["wq"], wq)


def test_one_row_of_a_wider_buffer(M):
    """A single token's codes, activations, output and logits as a row of a buffer of any stride."""
    lin, wq = product(M, 70, 200)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    codes = torch.randint(-127, 128, (8, 300), generator=g, device="cuda", dtype=torch.int8)
    sx = torch.rand(1, generator=g, device="cuda")
    y = [torch.full((4, n), 7.0, dtype=torch.bfloat16, device="cuda") for n in (70, 77)]
    M.moe_w8a8_linear_forward_codes(lin, codes[:1, :200].contiguous(), sx, 1, y[0])
    M.moe_w8a8_linear_forward_codes(lin, codes[:1, :200], sx, 1, y[1])
    assert torch.equal(y[0][0], y[1][0, :70]) and (y[1][0, 70:] == 7).all() and (y[1][1:] == 7).all()
    x = torch.randn(8, 203, generator=g, device="cuda").bfloat16()
    ws = torch.empty(M.moe_w8a8_linear_workspace_size(lin, 1), dtype=torch.uint8, device="cuda")
    M.moe_w8a8_linear_forward(lin, x[:1, :200].contiguous(), 1, y[0], ws)
    M.moe_w8a8_linear_forward(lin, x[:1, :200], 1, y[1], ws)
    assert torch.equal(y[0][0], y[1][0, :70])
    q = [torch.empty(1, 208, dtype=torch.int8, device="cuda"), torch.full((2, 300), 9, dtype=torch.int8, device="cuda")]
    s = [torch.empty(1, device="cuda"), torch.empty(1, device="cuda")]
    for i in range(2):
        M.moe_w8a8_block_norm(M.make_norm_config(200), 1, x=x[:1, :200], w_pre=torch.ones(200, device="cuda"), xq=q[i], sx=s[i])
    assert torch.equal(q[0][0, :200], q[1][0, :200]) and (q[1][0, 200:] == 9).all() and (q[1][1] == 9).all()
    assert torch.equal(s[0], s[1])
    u, token = torch.rand(1, generator=g, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    M.moe_w8a8_sample(x[:1, :200].contiguous(), u, token[:1])
    M.moe_w8a8_sample(x[:1, :200], u, token[1:])
    assert token[0] == token[1]
