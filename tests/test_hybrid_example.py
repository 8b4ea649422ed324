"""The hybrid decoder example's kept workspaces, without a GPU: each call gets one of its size."""
import importlib.util
import os

import pytest
import torch

import gated_deltanet_linear_05_gb300 as gdn
from gated_deltanet_linear_05_gb300 import build as gdn_build

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_decoder.py")


@pytest.fixture
def example(monkeypatch):
    gdn_build.build()
    spec = importlib.util.spec_from_file_location("hybrid_decoder_cpu", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    monkeypatch.setattr(gdn, "gdn_attn_workspace", lambda n, t, hq, hkv, d, prefix_len=0: torch.zeros(
        gdn.gdn_attn_workspace_size(gdn.make_attn_shape(n, t, hq, hkv, d, prefix_len=prefix_len)), dtype=torch.uint8,
        device="meta"))
    return m


def _need(layer, n, tokens, prefix):
    return gdn.gdn_attn_workspace_size(gdn.make_attn_shape(n, tokens, layer.hq, layer.hkv, layer.d, prefix_len=prefix))


@pytest.mark.parametrize("order", [(0, 1), (1, 0)])
def test_plain_and_prefixed_batches_of_one_size(example, order):
    model = example.Model(device="cpu")
    layer = next(l for l in model.layers if l.kind == "attention")
    plain = example.Batch(model, 1, 40)
    plain.length = 33
    prefixed = example.Batch(model, 1, 40, plain)
    for i in order:
        batch, prefix = ((plain, 0), (prefixed, 33))[i]
        for tokens in (33, 1):
            assert model.workspace("attention", batch, tokens, layer).numel() >= _need(layer, 1, tokens, prefix)


def test_longer_prefix_of_the_same_batch_size(example):
    """Another system prompt's batch of the same size."""
    model = example.Model(device="cpu", pages=4000)
    layer = next(l for l in model.layers if l.kind == "attention")
    for length in (33, 20000, 33):
        head = example.Batch(model, 1, length)
        head.length = length
        batch = example.Batch(model, 3, 40, head)
        assert model.workspace("attention", batch, 3, layer).numel() >= _need(layer, 3, 3, length)
