"""The example block: training lowers its loss, decoding answers as the packed pass does."""
import importlib.util
import pathlib

import numpy as np
import pytest
import torch

from gpu_util import REL_FRO, f64, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    need_gpu()
    path = pathlib.Path(__file__).resolve().parent.parent / "examples" / "train_block.py"
    spec = importlib.util.spec_from_file_location("train_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("state_bits", [8, 32])
def test_training_lowers_the_loss(example, state_bits):
    losses, _ = example.train([100, 1, 155], 12, state_bits=state_bits)
    assert np.isfinite(losses).all()
    assert losses[-1] < losses[0]


def test_decoding_answers_as_the_packed_pass(example):
    lens = [2, 130, 33]
    w = example.Weights(2)
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randn(n, w.cfg.d, generator=g).to(torch.bfloat16).cuda() for n in lens]
    _, one = example.decode(w, prompts, slots=5)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    block = example.Block(w, sum(lens), 3, max(lens), backward=False)
    block.forward(torch.cat(prompts), cu)
    last = (cu[1:] - 1).long()
    ref, got = f64(block.mixer.o[last]), f64(one.mixer.o)
    assert np.linalg.norm(got - ref) <= 2 * REL_FRO * np.linalg.norm(ref)
    assert int(one.mixer.err) == 0 and int(block.mixer.err) == 0


def test_seeds_make_other_weights_of_the_same_sizes(example):
    for kind in (example.Weights, example.ScanWeights):
        a, b, c = kind(0), kind(3), kind(3)
        assert a.moe["Wr"].shape == b.moe["Wr"].shape and not torch.equal(a.moe["Wr"], b.moe["Wr"])
        assert all(torch.equal(b.moe[n], c.moe[n]) for n in ("Wr", "W13", "W_up"))
    losses, _ = example.train([20, 12], 2, seed=7)
    assert len(losses) == 2
