"""spec_verify_logprobs at every temperature that it takes, from fp32's smallest to its largest."""
import math

import pytest
import torch

from test_gpu_logprobs import BF, DEV, FP32, check, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_verification_verify_gb300 import _build

    _build.build()
    torch.cuda.set_device(DEV)


def fp32(x):
    return float(torch.tensor(x, dtype=torch.float32))


@pytest.mark.parametrize("dtype", [BF, FP32])
@pytest.mark.parametrize("T", [1e-40, 1e-38, 1e-37, 1e-30, 1e-20, 1e-10, 3e-9, 1e-6, 1e-3, 1e3, 1e10, 1e20, 9e26, 2e27, 5e28,
                               1e30, 1e35, 2.9e38])
@pytest.mark.parametrize("V", [9001, 128256])
def test_temperatures(dtype, T, V):
    """Masks of -inf have no part at any temperature; masks of the type's lowest value have the part that they
    have.  The largest logit is 0 (twice) in some rows and large in others."""
    T = fp32(T)
    low = torch.finfo(dtype).min
    x, tok = rows(1, 6, V, dtype, seed=31)
    g = torch.Generator(device=DEV)
    g.manual_seed(32)
    hide = torch.rand((V,), generator=g, device=DEV) < 0.5
    hide[:4] = torch.tensor([False, False, True, False], device=DEV)
    x[0, 0] -= x[0, 0].max()
    x[0, 0, 0] = x[0, 0, 1] = 0.0
    x[0, 1] = x[0, 0]
    x[0, 1, hide] = -math.inf
    x[0, 2, hide] = -math.inf
    x[0, 3, hide] = low
    x[0, 4] = 7.5
    x[0, 5] = -math.inf
    x[0, 5, 3] = -2.5
    tok[0] = torch.tensor([1, 0, 3, 3, V - 1, 3])
    check(x, tok, 5, temperature=T)
    check(x, tok, 0, temperatures=torch.full((1,), T, device=DEV))


@pytest.mark.parametrize("V", [9001, 128256])
def test_steps_of_large_logits(V):
    """Two values a step of fp32 apart at a size where the logits' products with the scale are whole numbers:
    tens of thousands of equal terms, which add up without bias."""
    x = torch.full((1, 3, V), 2.0e7 - 2.0, device=DEV)
    x[0, :, 5] = 2.0e7
    x[0, 2, ::2] = -math.inf
    check(x, torch.tensor([[5, 6, 7]], dtype=torch.int32, device=DEV), 3)
