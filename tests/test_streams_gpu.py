"""A stream that is not torch's, known by its handle alone, and torch's own
kinds of stream: the plain calls take each."""

import types

import pytest
import torch

import attention_distillation_kl_gb300 as skl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["torch", "external", "handle", "default", "handle of the default"])
def test_kinds_of_stream(kind):
    g = torch.Generator().manual_seed(4)
    x = [torch.randn((1, 2, 200, 64), generator=g).to(torch.bfloat16).cuda() for _ in range(4)]
    want = [t.clone() for t in skl.streamkl_fwd(*x, 0.125, True)]
    torch.cuda.synchronize()
    own = torch.cuda.Stream()
    s = {"torch": own, "external": torch.cuda.ExternalStream(own.cuda_stream),
         "handle": types.SimpleNamespace(cuda_stream=own.cuda_stream), "default": torch.cuda.default_stream(),
         "handle of the default": types.SimpleNamespace(cuda_stream=torch.cuda.default_stream().cuda_stream)}[kind]
    for got in (skl.streamkl_fwd(*x, 0.125, True, stream=s), skl.streamkl_fwd(*x, 0.125, True, None, None, None, s),
                skl.streamkl_fwd_splitk(*x, 0.125, True, 1, stream=s)):
        torch.cuda.synchronize()
        assert all(torch.allclose(a, b, rtol=1e-5, atol=1e-5) for a, b in zip(got, want))
