"""Blocks whose memory moves: host-side checks that need no GPU."""
import pytest
import torch

import parameter_layout_collectives_amd as tide
from parameter_layout_collectives_amd import blocks as impl
from test_blocks_host import _Stub, stub_blocks


class _At(_Stub):
    """A stub with an address."""

    def __init__(self, at, *args, **kw):
        super().__init__(*args, **kw)
        self.at = at

    def data_ptr(self):
        return self.at


def test_pointers_follow_the_storage():
    q = tide.Blocks.empty(64, 1000, device="cpu")
    for t in (q.codes, q.scales):
        size = t.untyped_storage().nbytes()
        t.untyped_storage().resize_(0)
        assert q._ptrs == (q.codes.data_ptr(), q.scales.data_ptr()) and 0 in q._ptrs
        hold = torch.empty(size, dtype=torch.uint8)      # so that it does not come back by chance
        t.untyped_storage().resize_(size)
        assert q._ptrs == (q.codes.data_ptr(), q.scales.data_ptr()) and 0 not in q._ptrs
        del hold


def blocks_at(rows, cols, codes, scales):
    return tide.Blocks(_At(codes, (rows, -(-cols // 128) * 128), torch.uint8),
                       _At(scales, (rows, -(-cols // 512) * 4), torch.uint8), cols)


def test_calls_take_the_replaced_tensors(monkeypatch):
    calls = []
    monkeypatch.setattr(impl, "_call", lambda device, fn, *args: calls.append(args))
    x, w = blocks_at(4, 200, 1 << 20, 2 << 20), blocks_at(8, 200, 3 << 20, 4 << 20)
    out = _At(5 << 20, (4, 8), torch.bfloat16)
    tide.block_mm(x, w, out=out)
    w.codes = _At(6 << 20, (8, 256), torch.uint8)
    w.scales = _At(7 << 20, (8, 4), torch.uint8)
    x.codes.at = 8 << 20
    tide.block_mm(x, w, out=out)
    assert calls[0][:6] == (1 << 20, 2 << 20, 4, 3 << 20, 4 << 20, 8)
    assert calls[1][:6] == (8 << 20, 2 << 20, 4, 6 << 20, 7 << 20, 8)


def test_a_replacement_has_to_fit():
    q = stub_blocks(4, 200)
    u8 = torch.uint8
    for name, t, exc in [("codes", _Stub((4, 384), u8), ValueError),
                         ("codes", _Stub((5, 256), u8), ValueError),
                         ("codes", _Stub((4, 256), torch.int8), TypeError),
                         ("codes", _Stub((4, 256), u8, "cuda:1"), ValueError),
                         ("codes", _Stub((4, 256), u8, contiguous=False), ValueError),
                         ("scales", _Stub((4, 8), u8), ValueError),
                         ("scales", _Stub((5, 4), u8), ValueError)]:
        before = q.codes, q.scales
        with pytest.raises(exc):
            setattr(q, name, t)
        assert (q.codes, q.scales) == before
    for name, value in (("cols", 256), ("rows", 5), ("device", "cuda:1")):
        with pytest.raises(AttributeError):
            setattr(q, name, value)
    assert q.shape == (4, 200)


def test_views_follow_the_tensors():
    plan = tide.BlockPlan(tide.Plan([(64, 1000)], 2))
    q = tide.Blocks.empty(64, 1000, device="cpu")
    first = plan.views([q])
    assert [v.data_ptr() for v in first] == list(q._ptrs)
    for t in (q.codes, q.scales):
        size = t.untyped_storage().nbytes()
        t.untyped_storage().resize_(0)
        hold = torch.empty(size, dtype=torch.uint8)
        t.untyped_storage().resize_(size)
        del hold
    assert [v.data_ptr() for v in plan.views([q])] == list(q._ptrs)


def test_views_of_replaced_tensors(monkeypatch):
    monkeypatch.setattr(impl, "_words", lambda t: t.at)
    plan = tide.BlockPlan(tide.Plan([(8, 200)], 2))
    w = blocks_at(8, 200, 3 << 20, 4 << 20)
    assert plan.views([w]) == [3 << 20, 4 << 20]
    w.codes = _At(6 << 20, (8, 256), torch.uint8)
    assert plan.views([w]) == [6 << 20, 4 << 20]
    w.scales = _At(7 << 20, (8, 4), torch.uint8)
    assert plan.views([w]) == [6 << 20, 7 << 20]
