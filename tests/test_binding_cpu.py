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
