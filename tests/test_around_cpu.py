"""The operators around the MoE layer without a GPU: what the library and the binding refuse, before anything is
enqueued."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def M():
    from w8a8_quantized_moe_b200 import build
    build.build()
    import w8a8_quantized_moe_b200 as mod
    return mod


OK, ODD = 1 << 20, (1 << 20) + 2


def test_linear_refusals(M):
    L = M.lib()
    out = ctypes.c_void_p(5)
    good = M.make_linear_config(1000, 500)

    def prep(cfg=good, w=OK, bias=None, absmax=None, to=ctypes.byref(out)):
        return L.moe_w8a8_linear_prepare(None if cfg is None else ctypes.byref(cfg), w, bias, absmax, None, to)

    def codes(cfg=good, wq=OK, sw=OK, bias=None, inv_s=None, to=ctypes.byref(out)):
        return L.moe_w8a8_linear_prepare_codes(None if cfg is None else ctypes.byref(cfg), wq, sw, bias, inv_s, None, to)

    bad, shape = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED_SHAPE
    assert prep(None) == bad and prep(to=None) == bad and prep(w=None) == bad and out.value is None
    assert prep(w=ODD) == bad and prep(bias=ODD) == bad and prep(absmax=ODD) == bad
    assert codes(None) == bad and codes(to=None) == bad and codes(wq=None) == bad and codes(sw=None) == bad
    assert codes(sw=ODD) == bad and codes(bias=ODD) == bad and codes(inv_s=ODD) == bad
    for field, value, status in [("alpha", -0.1, bad), ("alpha", 1.1, bad), ("alpha", float("nan"), bad),
                                 ("in_dtype", 2, bad), ("out_dtype", -1, bad), ("n", 0, shape), ("k", 0, shape),
                                 ("n", M.MOE_LINEAR_MAX_N + 1, shape), ("k", M.MOE_LINEAR_MAX_K + 1, shape)]:
        c = M.make_linear_config(1000, 500)
        setattr(c, field, value)
        assert prep(c) == status and codes(c) == status, field
    assert L.moe_w8a8_linear_forward(None, OK, 500, 4, OK, 1000, OK, 1 << 20, None) == bad
    assert L.moe_w8a8_linear_forward_codes(None, OK, 512, OK, 4, OK, 1000, None) == bad
    assert L.moe_w8a8_linear_export(None, OK, OK, None, None) == bad
    assert L.moe_w8a8_linear_check_status(None, None) == bad
    assert L.moe_w8a8_linear_workspace_size(None, 4) == 0
    L.moe_w8a8_linear_destroy(None)


def norm_io(M, **kw):
    d = dict(b=OK, ldb=256, x=OK, ldx=256, w_pre=OK, x_out=OK, ldxo=256, n_out=OK, ldn=256)
    d.update(kw)
    io = M.moe_w8a8_norm_io()
    for k, v in d.items():
        setattr(io, k, v)
    return ctypes.byref(io)


def test_block_norm_refusals(M):
    L = M.lib()
    bad, shape = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED_SHAPE
    cfg = M.make_norm_config(256)
    call = lambda c, io, T=4: L.moe_w8a8_block_norm(ctypes.byref(c), io, T, None)  # noqa: E731
    assert L.moe_w8a8_block_norm(None, norm_io(M), 4, None) == bad
    assert L.moe_w8a8_block_norm(ctypes.byref(cfg), None, 4, None) == bad
    assert call(cfg, norm_io(M), -1) == bad
    assert call(cfg, norm_io(M), 0) == M.MOE_OK          # nothing to do, nothing enqueued
    for field, value, status in [("in_dtype", 3, bad), ("res_dtype", -1, bad), ("out_dtype", 2, bad), ("gate", 4, bad),
                                 ("gate", -1, bad), ("gate_sigmoid", 2, bad), ("eps", 0.0, bad), ("eps", -1.0, bad),
                                 ("eps", float("nan"), bad), ("eps", float("inf"), bad),
                                 ("residual_scale", float("inf"), bad), ("branch_scale", float("nan"), bad),
                                 ("weight_offset", float("nan"), bad), ("d", 0, shape),
                                 ("d", M.MOE_NORM_MAX_D + 1, shape)]:
        c = M.make_norm_config(256)
        setattr(c, field, value)
        assert call(c, norm_io(M)) == status, (field, value)
    for kw in [dict(b=None, x=None), dict(ldb=255), dict(ldx=100), dict(ldxo=255), dict(ldn=1), dict(b=OK + 1), dict(x=OK + 1),
               dict(x_out=OK + 1), dict(n_out=OK + 1), dict(w_pre=ODD), dict(w_post=ODD), dict(w_pre=None),
               dict(x_out=None, n_out=None), dict(xq=OK, ldq=256), dict(sx=OK), dict(xq=OK + 8, ldq=256, sx=OK),
               dict(xq=OK, ldq=264, sx=OK), dict(xq=OK, ldq=240, sx=OK), dict(xq=OK, ldq=256, sx=ODD), dict(inv_s=OK),
               dict(xq=OK, ldq=256, sx=OK, inv_s=ODD), dict(gate=OK), dict(b=None, w_post=OK), dict(ldb=1 << 60)]:
        assert call(cfg, norm_io(M, **kw)) == bad, kw
    for gate in (M.MOE_GATE_CHANNEL, M.MOE_GATE_TOKEN, M.MOE_GATE_ELEMENT):
        c = M.make_norm_config(256, gate=gate)
        assert call(c, norm_io(M)) == bad                # the gate is missing
        assert call(c, norm_io(M, gate=OK + 1, ldg=256)) == bad
        assert call(c, norm_io(M, gate=OK, ldg=256, b=None)) == bad
    assert call(M.make_norm_config(256, gate=M.MOE_GATE_ELEMENT), norm_io(M, gate=OK, ldg=255)) == bad


def test_sample_refusals(M):
    L = M.lib()
    bad, shape = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED_SHAPE

    def call(rows=4, vocab=1000, dtype=0, **kw):
        io = M.moe_w8a8_sample_io()
        for k, v in dict(dict(logits=OK, ld=1000, u=OK, token=OK), **kw).items():
            setattr(io, k, v)
        return L.moe_w8a8_sample(ctypes.byref(io), rows, vocab, dtype, None)

    assert L.moe_w8a8_sample(None, 4, 1000, 0, None) == bad
    assert call(rows=-1) == bad and call(dtype=2) == bad and call(dtype=-1) == bad
    assert call(vocab=0) == shape and call(vocab=M.MOE_SAMPLE_MAX_VOCAB + 1, ld=1 << 20) == shape
    assert call(rows=M.MOE_SAMPLE_MAX_ROWS + 1) == shape
    assert call(rows=0) == M.MOE_OK
    for kw in [dict(logits=None), dict(logits=OK + 2), dict(ld=999), dict(ld=-1), dict(u=None), dict(u=ODD), dict(token=None),
               dict(token=ODD), dict(prob=ODD), dict(temperature=ODD), dict(top_k=ODD), dict(top_p=ODD), dict(min_p=ODD),
               dict(allowed=OK, ld_allowed=31), dict(allowed=ODD, ld_allowed=32)]:
        assert call(**kw) == bad, kw


def test_binding_refuses_host_tensors(M):
    """The binding takes CUDA tensors only; it says so before it calls the library."""
    import torch
    lin = M.Linear(None, M.make_linear_config(16, 32), False)
    x, y = torch.zeros(2, 32, dtype=torch.bfloat16), torch.zeros(2, 16, dtype=torch.bfloat16)
    ws = torch.zeros(1024, dtype=torch.uint8)
    try:
        M.torch_device = M._device
        M._device = lambda: 0
        with pytest.raises(TypeError, match="x"):
            M.moe_w8a8_linear_forward(lin, x, 2, y, ws)
        with pytest.raises(TypeError, match="xq"):
            M.moe_w8a8_linear_forward_codes(lin, torch.zeros(2, 32, dtype=torch.int8), torch.zeros(2), 2, y)
        with pytest.raises(TypeError, match="b must"):
            M.moe_w8a8_block_norm(M.make_norm_config(32), 2, b=x, x_out=x)
        with pytest.raises(TypeError, match="logits"):
            M.moe_w8a8_sample(torch.zeros(2, 9), torch.zeros(2), torch.zeros(2, dtype=torch.int32))
    finally:
        M._device = M.torch_device
        del M.torch_device


def test_limits_match_the_header(M):
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_w8a8.h")).read()
    for name in ("MOE_LINEAR_MAX_N", "MOE_LINEAR_MAX_K", "MOE_NORM_MAX_D", "MOE_SAMPLE_MAX_VOCAB", "MOE_SAMPLE_MAX_ROWS"):
        value = re.search(rf"#define {name} (.+)", text).group(1)
        assert eval(value) == getattr(M, name), name


def test_the_norms_range_fits_fp32():
    """The largest values that the header allows leave the sum of squares of the longest row within fp32."""
    import os
    import re
    import numpy as np
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_w8a8.h")).read()
    part = re.sub(r"\s*\n \*\s*", " ", text[text.index("The norms around a block"):])
    bound = float(re.search(r"\|values\| up to (\d+e\d+)", part).group(1))
    longest = int(re.search(r"#define MOE_NORM_MAX_D (\d+)", text).group(1))
    assert longest * bound ** 2 < float(np.finfo(np.float32).max)
