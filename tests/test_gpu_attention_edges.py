"""Attention at the edges of what its description allows, on a B200: values that are not numbers, padding that holds
anything, loss-scaled FP16 gradients, saturated caps, strided outputs. Tolerances as in test_gpu_attention.py, with
what a test adds written beside it."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import operator_refs as R  # noqa: E402
from latent_diffusion_net_b200 import binding as B  # noqa: E402
from test_gpu_attention import call, compare, i32, inputs, packed, reference  # noqa: E402


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_documents_cut_anywhere_in_long_rows(d, causal):
    """Tiles of one document, tiles with a cut inside and tiles that nobody sees in turns, through many more steps than
    the documents' ring has places, in CTAs that take several units and end after any kind of step."""
    cuts = [[0, 130, 131, 700, 1280, 1900, 2600], [0, 1, 64, 1000, 1024, 2000, 2690]]
    n = 2700
    doc = torch.zeros(2, n, dtype=torch.int32, device="cuda")
    for b, at in enumerate(cuts):
        for i, c in enumerate(at):
            doc[b, c:] = (i * 5) % 7  # ids in no order
    q, k, v, do = inputs(2, n, n, 6, 2, d, "bf16", 75)
    kw = dict(causal=causal, q_doc=doc, k_doc=doc, k_lens=i32([n, 2650]))
    compare(call(q, k, v, do, **kw), reference(q, k, v, do, **kw), q.dtype)
