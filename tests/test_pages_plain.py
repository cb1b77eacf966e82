"""The plain forms that the page operators are tested against, checked by hand and
against each other, and the entry points' host-side refusals (no GPU needed)."""
import ctypes as C
import math

import pytest
import torch

import _pages as P


def test_seen_mask_chain_and_tree():
    L, T = 10, 4
    for t in range(T):
        assert P.seen_mask(L, T, None, t).tolist() == [p <= 6 + t for p in range(L)]
    chain = [(1 << (t + 1)) - 1 for t in range(T)]
    for t in range(T):  # a chain written as a tree
        assert P.seen_mask(L, T, chain, t).tolist() == P.seen_mask(L, T, None, t).tolist()
    tree = [1, 1 | 2, 1 | 4, 0]
    assert P.seen_mask(L, T, tree, 2).tolist() == [True] * 6 + [True, False, True, False]
    assert P.seen_mask(L, T, tree, 3).tolist() == [True] * 6 + [False] * 4
    assert P.seen_mask(3, 4, None, 0).tolist() == [False] * 3


def test_attention_closed_forms():
    kv = torch.randn(5, P.DIM, dtype=torch.float64)
    q = torch.zeros(2, P.DIM, dtype=torch.float64)
    keep = torch.tensor([True, False, True, True, False])
    out, lse, mass, _ = P.attention(q, kv, keep, 0.1)
    assert torch.allclose(out[0], kv[keep][:, :P.NOPE].mean(0))
    assert torch.allclose(mass[1], kv[keep][:, :P.NOPE].abs().mean(0))
    assert abs(float(lse[1]) - math.log(3)) < 1e-12
    out, lse, _, _ = P.attention(q, kv, torch.zeros(5, dtype=torch.bool), 0.1)
    assert not out.any() and bool((lse == -math.inf).all())


def test_select_plain():
    means = torch.zeros(6, P.DIM, dtype=torch.float64)
    means[:, 0] = torch.tensor([0.0, 5, 3, 5, 1, 2])
    q = torch.zeros(2, P.DIM, dtype=torch.float64)
    q[0, 0] = 1
    assert P.select(q, means, 6, 3, 0, 0) == [1, 2, 3]
    assert P.select(q, means, 6, 3, 1, 1) == [0, 1, 5]  # equal scores: the lower page
    assert P.select(q, means, 6, 2, 1, 1) == [0, 5]
    assert P.select(q, means, 2, 3, 1, 1) == [0, 1]
    q[1, 0] = -2  # the largest product of any head
    assert P.select(q, means, 6, 2, 0, 0) == [1, 3]
    q[0, 0] = -1
    assert P.select(q, means, 6, 1, 0, 0) == [0]


def test_quantise_plain():
    x = torch.zeros(4, P.DIM).to(torch.bfloat16)
    x[1, 3] = -7.0
    x[1, 5] = 3.5
    x[2, 0] = math.inf
    x[3, 0] = 2.0 ** -130
    codes, scale = P.quantise(x)
    assert float(scale[0]) == 2.0 ** -126 and not codes[0].float().any()
    assert float(scale[1]) == 7.0 / 448 and float(codes[1, 3].float()) == -448 and float(codes[1, 5].float()) == 224
    assert math.isnan(float(scale[2]))
    assert float(scale[3]) == 2.0 ** -126 and float(codes[3, 0].float()) == 2.0 ** -4


def test_entry_points_refuse_a_null_pool_and_plan_without_one():
    import __graft_entry__ as g
    g.build()
    import tiered_sparse_mla_gb300 as hs
    lib = hs.load()
    p = C.cast((C.c_int32 * 64)(), C.c_void_p)
    inval = hs.HS_ERR_INVALID_ARG
    assert lib.hs_append_rows(None, 1, 1, p, p, None, None, None) == inval
    assert lib.hs_page_means(None, 1, p, p, p, None) == inval
    assert lib.hs_select_pages(None, 1, 1, 16, 4, 1, 1, p, p, p, None, p, None, p, 1 << 20, None) == inval
    assert lib.hs_page_mla_decode(None, 1, 1, 16, 4, p, p, p, None, C.c_float(0.1), p, p, None, 0, None) == inval
    assert lib.hs_page_mla_decode_per_token(None, 1, 1, 16, 4, p, p, p, None, C.c_float(0.1), p, p, None, 0,
                                            None) == inval
    assert lib.hs_select_workspace_bytes(None, 4, 4) == 0
    assert lib.hs_page_decode_workspace_bytes(0, 1, 16, 4) == 0
    assert lib.hs_page_decode_workspace_bytes(1, 1, 16, 0) == 0
    assert lib.hs_page_decode_workspace_bytes(1, 8, 16, 2048) > 0


@pytest.mark.parametrize("devices", [1, 2])
def test_bindings_refuse_tensors_of_another_device(monkeypatch, devices):
    import tiered_sparse_mla_gb300 as hs

    class OnDevice(torch.Tensor):
        is_cuda = True
        device_index = 0

        def get_device(self):
            return self.device_index

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: devices)
    monkeypatch.setattr(hs, "_only_device", None)
    x = torch.zeros(3, dtype=torch.int32).as_subclass(OnDevice)
    for _ in range(2):  # the first look and the short one
        assert hs._arg("x", x, "int32", 3) == x.data_ptr()
        assert hs._ws(x) == (12, x.data_ptr())
    x.device_index = 1
    for call in (lambda: hs._arg("x", x, "int32", 3), lambda: hs._ws(x)):
        with pytest.raises(ValueError, match="device 1"):
            call()
    with pytest.raises(ValueError):
        hs._arg("x", torch.zeros(3, dtype=torch.int32), "int32", 3)
