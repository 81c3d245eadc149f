"""What the binding of the modified scores refuses before it reaches the
library: arguments that are no tensors."""

import types

import pytest
import torch

import attention_distillation_kl_gb300 as skl


@pytest.mark.parametrize("kw", [dict(causal=True, prefix=[3, 4]), dict(doc_q=[[0, 0]], doc_k=[[0, 0]]), dict(causal=True, prefix=3)])
def test_masks_that_are_no_tensors(kw):
    side = types.SimpleNamespace(rows=(2, 4, 8), keys=8, device=torch.device("cpu"))
    with pytest.raises(ValueError):
        skl._mod_call(side, side, kw.get("causal", False), kw.get("prefix"), kw.get("doc_q"), kw.get("doc_k"))


def test_a_workspace_that_is_no_tensor():
    with pytest.raises(ValueError):
        skl._mod_workspace(bytearray(64), 64, torch.device("cpu"), None)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(slopes=[0.5, 0.25]), dict(table=[[0.0] * 8] * 2), dict(slopes=0.5)])
def test_biases_that_are_no_tensors(kw):
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        skl.AttnSide(x, x, 0.125, **kw)
