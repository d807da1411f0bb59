"""Windows up to the largest number: as wide as the tokens, they leave the spans as they are."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_fine_nf4_amd as nf4  # noqa: E402

DEV = "cuda:0"


@pytest.mark.parametrize("window", [299, 300, 301, 2 ** 31, 2 ** 62, 2 ** 63 - 301, 2 ** 63 - 2, 2 ** 63 - 1])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("prefix", [None, [0, 2, 90, 100]])
def test_wide_windows(window, causal, prefix):
    M, docs = 300, [0, 1, 1, 70, 299]
    got = nf4.qlora_attn_spans(torch.tensor(docs, dtype=torch.int32, device=DEV), M,
                               None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device=DEV),
                               causal=causal, window=window)
    assert np.array_equal(got.cpu().numpy(), oracle.spans(docs, M, prefix, causal=causal, window=window))
