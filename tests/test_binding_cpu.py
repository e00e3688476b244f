"""The binding's own bookkeeping, without a GPU."""
import pytest


@pytest.fixture(scope="module")
def M():
    from w8a8_quantized_moe_b200 import build
    build.build()
    import w8a8_quantized_moe_b200 as mod
    return mod


def test_a_product_keeps_its_own_configuration(M, monkeypatch):
    """The caller's configuration may be changed for the next product: what the first handle's calls allocate and check
    goes by the sizes that it was prepared with."""
    import torch
    cfg = M.make_linear_config(48, 32)
    lin = M.Linear(None, cfg, True)
    cfg.n, cfg.k, cfg.in_dtype = 4, 2, M.MOE_F32
    assert (lin.cfg.n, lin.cfg.k, lin.cfg.in_dtype) == (48, 32, M.MOE_BF16)
    asked = []
    monkeypatch.setattr(M, "_device", lambda: 0)
    monkeypatch.setattr(M, "_stream", lambda s: None)
    monkeypatch.setattr(M, "lib", lambda: type("L", (), dict(moe_w8a8_linear_export=lambda *a: 0)))
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda size, dtype, device: asked.append(size) or empty(size, dtype=dtype))
    M.moe_w8a8_linear_export(lin)
    assert asked == [(48, 32), 48, 32]


def test_a_layer_keeps_its_own_configuration(M):
    """The sizes that a layer's calls check their tensors by are those that it was prepared with."""
    import torch
    cfg = M.make_config(256, 512, 8, 2, in_dtype=M.MOE_F32, out_dtype=M.MOE_F32)
    w = M.Weights(None, cfg)
    cfg.d, cfg.n_experts = 128, 4
    assert (w.cfg.d, w.cfg.n_experts, w.n_local) == (256, 8, 8)
    with pytest.raises(ValueError, match="x holds"):
        M.moe_w8a8_forward(w, torch.zeros(16 * 128), 16, None, None, torch.zeros(16 * 256), torch.zeros(16))


def test_the_stride_of_a_single_row_is_not_used(M):
    """One row of a wider buffer is taken like a row alone, whatever the buffer's stride: codes with a stride that is no
    multiple of 16 are not refused, activations off the 16-byte boundaries keep the wide accesses."""
    import torch
    for buffer in (torch.zeros(8, 300, dtype=torch.int8), torch.zeros(8, 201, dtype=torch.int8), torch.zeros(1, 200, dtype=torch.int8)):
        assert M._matrix(buffer[:, :200], 1, 200, "xq", torch.int8, -1) == (buffer.data_ptr(), 208)
        assert M._matrix(buffer, 1, 200, "xq", torch.int8, -1) == (buffer.data_ptr(), 208)
    two = torch.zeros(8, 300, dtype=torch.int8)
    assert M._matrix(two, 2, 200, "xq", torch.int8, -1) == (two.data_ptr(), 300)


def test_missing_tensors_are_named(M, monkeypatch):
    """A tensor that is missing or no tensor is refused by its name, like one of the wrong kind."""
    import torch
    monkeypatch.setattr(M, "_device", lambda: -1)       # the host, as the checks see it
    lin = M.Linear(None, M.make_linear_config(16, 32), False)
    x, y = torch.zeros(2, 32, dtype=torch.bfloat16), torch.zeros(2, 16, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="workspace"):
        M.moe_w8a8_linear_forward(lin, x, 2, y, None)
    with pytest.raises(TypeError, match="x must"):
        M.moe_w8a8_linear_forward(lin, None, 2, y, None)
    for logits, error in ((None, TypeError), ([[1.0]], TypeError), (torch.zeros(5), ValueError)):
        with pytest.raises(error, match="logits"):
            M.moe_w8a8_sample(logits, torch.zeros(2), torch.zeros(2, dtype=torch.int32))
