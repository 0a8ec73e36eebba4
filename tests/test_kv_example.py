"""The serving example's bookkeeping between steps, without a GPU."""
import importlib.util
import os

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load_example():
    spec = importlib.util.spec_from_file_location("paged_serving", os.path.join(ROOT, "examples", "paged_serving.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


def test_lengths_after_a_step_keep_a_refused_request():
    """Granted, idle, ended, refused, new and refused, new and granted: only the ended one starts again at 0."""
    i32 = dict(dtype=torch.int32)
    past = torch.tensor([20, 7, 33, 48, 0, 0], **i32)
    new = torch.tensor([1, 0, -1, 5, 9, 4], **i32)
    seq_lens = torch.tensor([21, 7, 0, 0, 0, 4], **i32)
    load_example().advance(past, new, seq_lens)
    assert past.tolist() == [21, 7, 0, 48, 0, 4] and past.dtype == torch.int32
