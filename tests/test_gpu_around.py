"""The operators around the MoE layer together: a decode step of a small model, from the hidden states to the next
token; calls at once on two streams; what live handles refuse."""
import numpy as np
import pytest
import torch

from tests import around_ref as R

pytestmark = pytest.mark.gpu
U32, UBF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def M():
    import w8a8_quantized_moe_b200 as mod
    torch.cuda.set_device(0)
    return mod


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


class Step:
    """x -> norm, codes -> projection -> residual add, norm -> MoE layer -> residual add with a gate, norm after the
    block -> final norm -> LM head -> token.  Buffers are made once, as a serving program would."""

    def __init__(self, M, T, d=256, f=512, E=8, k=2, vocab=5000, seed=0):
        self.M, self.T, self.d, self.vocab = M, T, d, vocab
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
        self.absmax = torch.zeros(d, device="cuda")
        M.moe_w8a8_calibrate_absmax(r(512, d), self.absmax)
        self.proj = M.moe_w8a8_linear_prepare(M.make_linear_config(d, d), r(d, d, std=d ** -0.5), r(d, std=0.1), self.absmax)
        self.head = M.moe_w8a8_linear_prepare(M.make_linear_config(vocab, d, out_dtype=M.MOE_F32), r(d, vocab, std=0.3))
        self.moe = M.moe_w8a8_prepare(M.make_config(d, f, E, k), r(E, d, f, std=d ** -0.5), r(E, d, f, std=d ** -0.5),
                                      r(E, f, d, std=f ** -0.5), r(d, E, std=d ** -0.5), self.absmax)
        self.inv_s = M.moe_w8a8_linear_export(self.proj)["inv_s"]
        self.w = [torch.rand(d, generator=g, device="cuda") + 0.5 for _ in range(4)]
        self.gate = r(d)
        self.pre = M.make_norm_config(d)
        self.mid = M.make_norm_config(d, gate=M.MOE_GATE_CHANNEL, gate_sigmoid=True, residual_scale=1.0, branch_scale=0.5)
        b = lambda n, dt=torch.bfloat16: torch.empty(T, n, dtype=dt, device="cuda")  # noqa: E731
        self.x, self.xq, self.sx = b(d), b(d, torch.int8), torch.empty(T, device="cuda")
        self.a, self.x1, self.n1, self.m, self.x2, self.n2, self.logits = b(d), b(d), b(d), b(d), b(d), b(d), b(vocab, torch.float32)
        self.u, self.token, self.prob = torch.empty(T, device="cuda"), torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, device="cuda")
        self.top_p = torch.full((T,), 0.9, device="cuda")
        self.top_k = torch.full((T,), 40, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(M.moe_w8a8_workspace_size(self.moe, T), dtype=torch.uint8, device="cuda")
        self.ws_head = torch.empty(M.moe_w8a8_linear_workspace_size(self.head, T), dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        M, T = self.M, self.T
        M.moe_w8a8_block_norm(self.pre, T, x=self.x, w_pre=self.w[0], inv_s=self.inv_s, xq=self.xq, sx=self.sx, stream=stream)
        M.moe_w8a8_linear_forward_codes(self.proj, self.xq, self.sx, T, self.a, stream=stream)
        M.moe_w8a8_block_norm(self.pre, T, b=self.a, x=self.x, w_pre=self.w[1], x_out=self.x1, n_out=self.n1, stream=stream)
        M.moe_w8a8_forward(self.moe, self.n1, T, None, None, self.m, self.ws, stream=stream)
        M.moe_w8a8_block_norm(self.mid, T, b=self.m, x=self.x1, gate=self.gate, w_post=self.w[2], w_pre=self.w[3], x_out=self.x2,
                              n_out=self.n2, stream=stream)
        M.moe_w8a8_linear_forward(self.head, self.n2, T, self.logits, self.ws_head, stream=stream)
        M.moe_w8a8_sample(self.logits, self.u, self.token, top_k=self.top_k, top_p=self.top_p, prob=self.prob, stream=stream)

    def outputs(self):
        return [t.clone() for t in (self.a, self.x1, self.n1, self.m, self.x2, self.n2, self.logits, self.token, self.prob)]

    def feed(self, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.x.copy_(torch.randn(self.T, self.d, generator=g, device="cuda") * 2)
        self.u.copy_(torch.rand(self.T, generator=g, device="cuda"))


@pytest.mark.parametrize("T", [1, 5, 300])
def test_decode_step(M, T):
    """Each stage against its definition, on the inputs that the stage before it produced."""
    s = Step(M, T)
    s.feed(7)
    s.run()
    torch.cuda.synchronize()
    M.moe_w8a8_linear_check_status(s.proj)
    M.moe_w8a8_linear_check_status(s.head)
    M.moe_w8a8_check_status(s.moe)
    eps = np.float64(np.float32(1e-6))
    x, w = host(s.x), [host(v) for v in s.w]
    f32 = lambda v: v.astype(np.float32)  # noqa: E731
    # the codes of norm(x), and the projection that reads them
    q, sc = R.quantize_rows(f32(x) * f32(w[0]) * f32(host(s.inv_s)))
    assert np.array_equal(s.xq.cpu().numpy(), q)
    sx = host(s.sx)
    assert (np.abs(sx - sc / R.rms(x, eps)[:, 0]) <= 20 * U32 * sx).all()
    got = M.moe_w8a8_linear_export(s.proj)
    wq, sw = got["wq"].cpu().numpy(), got["sw"].cpu().numpy()
    acc = q.astype(np.float64) @ wq.astype(np.float64).T
    p = acc * sx[:, None] * sw.astype(np.float64)
    # (the bias is the handle's: the difference to the product has to be one row for all tokens)
    d = host(s.a) - p
    assert (np.abs(d - np.median(d, axis=0)) <= 2.02 * UBF * (np.abs(host(s.a)) + np.abs(p).max(0)) + 1e-6).all()
    # residual add and norm; the layer on it; the gated norm after the block
    x1 = x + host(s.a)
    assert (np.abs(host(s.x1) - x1) <= 1.01 * UBF * np.abs(x1) + 1e-30).all()
    n1 = host(s.x1) / R.rms(host(s.x1), eps) * w[1]
    assert (np.abs(host(s.n1) - n1) <= 1.02 * UBF * np.abs(n1) + 1e-30).all()
    y = torch.empty_like(s.m)
    M.moe_w8a8_forward(s.moe, s.n1, T, None, None, y, s.ws)
    assert torch.equal(y, s.m) and torch.isfinite(y.float()).all() and y.float().abs().max() > 0
    m = host(s.m)
    br = 0.5 * (m / R.rms(m, eps) * w[2]) / (1 + np.exp(-host(s.gate)))
    x2 = host(s.x1) + br
    assert (np.abs(host(s.x2) - x2) <= 1.01 * UBF * np.abs(x2) + 40 * U32 * (np.abs(host(s.x1)) + np.abs(br))).all()
    n2 = host(s.x2) / R.rms(host(s.x2), eps) * w[3]
    assert (np.abs(host(s.n2) - n2) <= 1.02 * UBF * np.abs(n2) + 1e-30).all()
    # logits and token
    got = M.moe_w8a8_linear_export(s.head)
    q, sc = R.quantize_rows(f32(host(s.n2)))
    ref, mag = R.linear(q, sc, got["wq"].cpu().numpy(), got["sw"].cpu().numpy())
    assert (np.abs(host(s.logits) - ref) <= 1.01 * 3 * U32 * mag + 1e-37).all()
    want, pr = R.sample(s.logits.cpu().numpy(), s.u.cpu().numpy(), top_k=s.top_k.cpu().numpy(), top_p=s.top_p.cpu().numpy())
    assert np.array_equal(s.token.cpu().numpy(), want)
    assert np.allclose(s.prob.cpu().numpy(), pr, rtol=1e-6)


def test_step_in_a_graph(M):
    """The whole step captured once and replayed on new inputs equals the step run call by call."""
    s = Step(M, 6)
    want = []
    for seed in (1, 2, 3):
        s.feed(seed)
        s.run()
        want.append(s.outputs())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for i, seed in ((2, 3), (0, 1), (1, 2), (1, 2)):
        s.feed(seed)
        s.token.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(s.outputs(), want[i]):
            assert torch.equal(a, b)


def test_two_streams_at_once(M):
    """Steps of their own buffers, many at once on two streams and interleaved, one of them replayed from a graph."""
    steps = [Step(M, 3, seed=5), Step(M, 40, seed=6)]
    want = []
    for s in steps:
        s.feed(11)
        s.run()
        want.append(s.outputs())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for s, st in zip(steps, streams):
            s.run(st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps[0].run()
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            graph.replay()
        steps[1].run(streams[1])
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        for a, b in zip(s.outputs(), w):
            assert torch.equal(a, b)


def test_one_handle_on_two_streams(M):
    """One product's handle serves two streams at once; each call has its own workspace and outputs."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    lin = M.moe_w8a8_linear_prepare_codes(M.make_linear_config(700, 512),
                                          torch.randint(-127, 128, (700, 512), generator=g, device="cuda", dtype=torch.int8),
                                          torch.rand(700, generator=g, device="cuda"))
    runs = []
    for T in (2, 33, 400):
        x = torch.randn(T, 512, generator=g, device="cuda").bfloat16()
        y = torch.empty(T, 700, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(M.moe_w8a8_linear_workspace_size(lin, T), dtype=torch.uint8, device="cuda")
        M.moe_w8a8_linear_forward(lin, x, T, y, ws)
        runs.append((T, x, y, ws, y.clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(30):
        for (T, x, y, ws, _w), st in zip(runs, streams):
            M.moe_w8a8_linear_forward(lin, x, T, y, ws, stream=st)
    torch.cuda.synchronize()
    for _T, _x, y, _ws, w in runs:
        assert torch.equal(y, w)


def test_refusals_of_live_handles(M):
    """What is refused once there is a handle; nothing is enqueued, outputs stay as they were."""
    k, n, T = 100, 60, 4
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    lin = M.moe_w8a8_linear_prepare_codes(M.make_linear_config(n, k), z(n, k, dt=torch.int8), z(n, dt=torch.float32))
    x, y = z(T, k), torch.full((T, n), 3.0, dtype=torch.bfloat16, device="cuda")
    xq, sx = z(T, 112, dt=torch.int8), z(T, dt=torch.float32)
    ws = z(M.moe_w8a8_linear_workspace_size(lin, T), dt=torch.uint8)
    L, h = M.lib(), lin.handle
    p = lambda t: t.data_ptr()  # noqa: E731
    bad = M.MOE_ERR_INVALID_ARG
    fwd = lambda x_=p(x), ldx=k, T_=T, y_=p(y), ldy=n, w_=p(ws), nb=ws.numel(): L.moe_w8a8_linear_forward(  # noqa: E731
        h, x_, ldx, T_, y_, ldy, w_, nb, None)
    cod = lambda q_=p(xq), ldq=112, s_=p(sx), T_=T, y_=p(y), ldy=n: L.moe_w8a8_linear_forward_codes(  # noqa: E731
        h, q_, ldq, s_, T_, y_, ldy, None)
    assert fwd(x_=None) == bad and fwd(y_=None) == bad and fwd(w_=None) == bad and fwd(ldx=k - 1) == bad
    assert fwd(ldy=n - 1) == bad and fwd(T_=-1) == bad and fwd(x_=p(x) + 1) == bad and fwd(y_=p(y) + 1) == bad
    assert fwd(w_=p(ws) + 16) == bad
    assert fwd(nb=ws.numel() - 1) == M.MOE_ERR_WORKSPACE_TOO_SMALL
    assert cod(q_=None) == bad and cod(q_=p(xq) + 8) == bad and cod(ldq=104) == bad and cod(ldq=96) == bad
    assert cod(s_=None) == bad and cod(s_=p(sx) + 2) == bad and cod(y_=None) == bad and cod(ldy=n - 1) == bad and cod(T_=-1) == bad
    assert fwd(T_=0) == M.MOE_OK and cod(T_=0) == M.MOE_OK
    assert L.moe_w8a8_linear_export(h, None, None, p(sx), None) == bad        # no smoothing in this handle
    torch.cuda.synchronize()
    assert (y == 3).all()
    M.moe_w8a8_linear_check_status(lin)
    with pytest.raises(ValueError, match="x must be"):
        M.moe_w8a8_linear_forward(lin, x, T + 1, y, ws)
    with pytest.raises(ValueError, match="y must be"):
        M.moe_w8a8_linear_forward(lin, x, T, y[:, :-1], ws)
    with pytest.raises(ValueError, match="contiguous rows"):
        M.moe_w8a8_linear_forward(lin, z(k, T).T, T, y, ws)
    with pytest.raises(ValueError, match="apart"):
        M.moe_w8a8_linear_forward(lin, z(1, k).expand(T, k), T, y, ws)
    with pytest.raises(TypeError, match="x must be torch.bfloat16"):
        M.moe_w8a8_linear_forward(lin, x.float(), T, y, ws)
    with pytest.raises(ValueError, match="sx holds"):
        M.moe_w8a8_linear_forward_codes(lin, xq, sx[:2], T, y)
    with pytest.raises(M.MoeError):
        M.moe_w8a8_linear_forward_codes(lin, z(T, 104, dt=torch.int8), sx, T, y)
    with pytest.raises(ValueError, match="w_pre holds"):
        M.moe_w8a8_block_norm(M.make_norm_config(k), T, x=x, w_pre=sx, n_out=x)
    with pytest.raises(ValueError, match="u holds"):
        M.moe_w8a8_sample(z(4, 50, dt=torch.float32), sx[:3], z(4, dt=torch.int32))
    with pytest.raises(ValueError, match="allowed must be"):
        M.moe_w8a8_sample(z(4, 50, dt=torch.float32), sx, z(4, dt=torch.int32), allowed=z(4, 1, dt=torch.int32))
    # an empty batch is no call
    M.moe_w8a8_sample(z(0, 50, dt=torch.float32), z(0, dt=torch.float32), z(0, dt=torch.int32))


def test_offsets_past_32_bits(M):
    """Rows so far apart that an element's offset passes 32 bits give what neighbouring rows give."""
    T, k, n, V, far = 3, 320, 200, 3000, (1 << 30) + 64
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    lin = M.moe_w8a8_linear_prepare_codes(M.make_linear_config(n, k),
                                          torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8),
                                          torch.rand(n, generator=g, device="cuda"))
    wide = torch.empty(T * far, dtype=torch.bfloat16, device="cuda")
    at = lambda cols, off=0: wide.as_strided((T, cols), (far, 1), off)  # noqa: E731
    x = torch.randn(T, k, generator=g, device="cuda").bfloat16()
    ws = torch.empty(M.moe_w8a8_linear_workspace_size(lin, 400), dtype=torch.uint8, device="cuda")
    y = torch.empty(T, n, dtype=torch.bfloat16, device="cuda")
    M.moe_w8a8_linear_forward(lin, x, T, y, ws)
    at(k).copy_(x)
    M.moe_w8a8_linear_forward(lin, at(k), T, at(n, 1024), ws)
    assert torch.equal(at(n, 1024), y)
    # codes that far apart, through the tensor maps
    codes = torch.empty(T * far, dtype=torch.int8, device="cuda").as_strided((T, k), (far, 1))
    sx = torch.empty(T, device="cuda")
    cfg = M.make_norm_config(k)
    near = torch.empty(T, k, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    w = torch.rand(k, generator=g, device="cuda") + 0.5
    nn = torch.empty(T, k, dtype=torch.bfloat16, device="cuda")
    M.moe_w8a8_block_norm(cfg, T, b=x, x=x, w_pre=w, n_out=nn, xq=near[0], sx=near[1])
    M.moe_w8a8_block_norm(cfg, T, b=at(k), x=at(k), w_pre=w, n_out=at(k, 4096), xq=codes, sx=sx)
    assert torch.equal(at(k, 4096), nn) and torch.equal(codes, near[0]) and torch.equal(sx, near[1])
    M.moe_w8a8_linear_forward_codes(lin, near[0], near[1], T, y)
    M.moe_w8a8_linear_forward_codes(lin, codes, sx, T, at(n, 8192))
    assert torch.equal(at(n, 8192), y)
    # rows off every boundary, and the logits
    odd = wide.as_strided((T, k), (far - 1, 1), 1)
    odd.copy_(x)
    n_odd, n_near = torch.empty_like(nn), torch.empty(T, k + 1, dtype=torch.bfloat16, device="cuda")[:, 1:]
    M.moe_w8a8_block_norm(cfg, T, b=odd, x=odd, w_pre=w, n_out=n_odd)
    M.moe_w8a8_block_norm(cfg, T, b=x, x=x, w_pre=w, n_out=n_near)      # the same accesses, rows next to each other
    assert torch.equal(n_odd, n_near)
    logits = torch.randn(T, V, generator=g, device="cuda").bfloat16()
    at(V, 16384).copy_(logits)
    u, p = torch.rand(T, generator=g, device="cuda"), torch.full((T,), 0.7, device="cuda")
    tok = torch.empty(2, T, dtype=torch.int32, device="cuda")
    M.moe_w8a8_sample(logits, u, tok[0], top_p=p)
    M.moe_w8a8_sample(at(V, 16384), u, tok[1], top_p=p)
    assert torch.equal(tok[0], tok[1])
