"""The binding of the paged-cache operators: numbers that the C interface cannot hold, vectors that overlap."""
import pytest
import torch

import rank_adapter_gemm_build_amd as rx

BF, I32 = torch.bfloat16, torch.int32


class _NoCalls:
    def __getattr__(self, name):
        raise AssertionError(f"the library was called: {name}")


def _object(cls, **kw):
    o = object.__new__(cls)
    o.__dict__.update(handle=0, **kw)
    return o


def _cache():
    return rx.KVCache(torch.zeros(4, 16, 2, 32, dtype=BF), torch.zeros(4, 16, 2, 32, dtype=BF))


def _far(rows, width, dtype, stride):
    """Rows `stride` elements apart, without their memory."""
    return torch.empty_strided((rows, width), (stride, 1), dtype=dtype, device="meta")


ATTENTION = dict(device=0, num_q_heads=4, num_kv_heads=2, head_dim=32)


@pytest.mark.parametrize("change", [dict(q=_far(3, 128, BF, 2 ** 32 + 128)), dict(out=_far(3, 128, BF, 2 ** 31)),
                                    dict(block_table=_far(2, 4, I32, 2 ** 32 + 4))])
def test_row_strides_past_31_bits_are_refused(monkeypatch, change):
    monkeypatch.setattr(rx.kv, "lib", _NoCalls())
    args = dict(q=torch.zeros(3, 128, dtype=BF), out=torch.zeros(3, 128, dtype=BF), block_table=torch.zeros(2, 4, dtype=I32))
    args.update(change)
    with pytest.raises(ValueError, match="row stride"):
        rx.paged_attention(_object(rx.Attention, **ATTENTION), args["q"], _cache(), args["block_table"], torch.zeros(2, dtype=I32),
                           torch.zeros(3, dtype=I32), args["out"])


def test_qkv_row_stride_past_31_bits_is_refused(monkeypatch):
    monkeypatch.setattr(rx.kv, "lib", _NoCalls())
    with pytest.raises(ValueError, match="row stride"):
        rx.rotary_append(_object(rx.Rotary, device=0, rot_dim=32, interleaved=False), _far(3, 256, BF, 2 ** 32 + 256), 4,
                         torch.zeros(3, dtype=I32), torch.zeros(3, dtype=I32), torch.zeros(3, 128, dtype=BF), _cache())


def test_the_stride_of_a_single_row_is_never_used():
    assert rx.kv._rows(_far(1, 128, BF, 2 ** 33 + 8), BF, 1, 128, "q")[1] == 128
    assert rx.kv._rows(_far(1, 20, BF, 1), BF, 1, 20, "q")[1] == 24
    assert rx.kv._table(_far(1, 4, I32, 2 ** 33), 1)[1:] == (4, 4)


@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32 + 5, 5 - 2 ** 32])
def test_windows_past_31_bits_are_refused(monkeypatch, window):
    """2^32 + 5 would arrive as 5."""
    monkeypatch.setattr(rx.kv, "lib", _NoCalls())
    with pytest.raises(ValueError, match="window"):
        rx.paged_attention(_object(rx.Attention, **ATTENTION), torch.zeros(3, 128, dtype=BF), _cache(), torch.zeros(2, 4, dtype=I32),
                           torch.zeros(2, dtype=I32), torch.zeros(3, dtype=I32), torch.zeros(3, 128, dtype=BF), window=window)


def test_sizes_past_31_bits_are_refused(monkeypatch):
    monkeypatch.setattr(rx.kv, "lib", _NoCalls())
    with pytest.raises(ValueError, match="max_tokens"):
        rx.Attention(0, 4, 2 ** 32 + 8, 4, 2, 32)
    plan = _object(rx.PagePlan, device=0, max_seqs=4, max_tokens=8, _out=[0] * 5)
    with pytest.raises(ValueError, match="page_size"):
        rx.page_plan(plan, torch.zeros(3, dtype=I32), torch.zeros(3, dtype=I32), 8, torch.zeros(8, dtype=I32), torch.zeros(4, dtype=I32),
                     torch.zeros(3, 4, dtype=I32), 2 ** 32 + 16)


@pytest.mark.parametrize("which,at", [("past", 0), ("past", 2), ("new", 0), ("new", 1)])
def test_lengths_that_the_plan_itself_writes_are_refused(monkeypatch, which, at):
    """A step's workgroups read past_lens and new_lens while another writes seq_lens."""
    monkeypatch.setattr(rx.kv, "lib", _NoCalls())
    out = {k: torch.zeros(n, dtype=I32) for k, n in dict(seq_lens=5, query_start=6, positions=8, slots=8, meta=8).items()}
    plan = _object(rx.PagePlan, device=0, max_seqs=5, max_tokens=8, _out=[t.data_ptr() for t in out.values()], **out)
    lens = dict(past=torch.zeros(3, dtype=I32), new=torch.zeros(3, dtype=I32))
    lens[which] = plan.seq_lens[at:at + 3]
    with pytest.raises(ValueError, match="overlap"):
        rx.page_plan(plan, lens["past"], lens["new"], 8, torch.zeros(8, dtype=I32), torch.zeros(4, dtype=I32),
                     torch.zeros(3, 4, dtype=I32), 16)
