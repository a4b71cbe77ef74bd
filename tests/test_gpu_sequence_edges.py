"""GPU: the sequence operators' calls at the edges: every kernel that the dispatch chooses, outputs of both types,
values at the ends of the types' ranges, bad offsets between guards."""
import pytest
import torch

from tests import seq_reference as R
from tests.test_gpu_sequence import BF16, F32, G, cu_of, rows  # noqa: F401  (G: the fixture)

pytestmark = pytest.mark.gpu


# One, two and more than two strips of 16 columns per CU of 256: a forward kernel each (fp32 inputs share the last two)
STRIPS = [([70, 130], 1, 2, 48, 48), ([70, 1, 64, 90] * 3, 2, 4, 112, 112), ([200, 64, 3] * 10, 2, 4, 128, 96)]


@pytest.mark.parametrize("lengths,hk,hv,dk,dv", STRIPS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_packed_forward_bf16_output_is_the_fp32_output_rounded(G, lengths, hk, hv, dk, dv, dtype):  # noqa: F811
    """The type of the output decides its one rounding and nothing before it."""
    x = rows(sum(lengths), hk, hv, dk, dv, dtype, 71)
    S0 = torch.randn(len(lengths), hv, dk, dv, generator=torch.Generator().manual_seed(72)).cuda()
    a, Sa = G.packed_forward(*x, cu_of(lengths), S0)
    b, Sb = G.packed_forward(*x, cu_of(lengths), S0, out_dtype=BF16)
    assert torch.equal(a.to(BF16), b) and torch.equal(Sa, Sb)
