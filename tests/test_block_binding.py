"""What the binding of the operators around the layers refuses, with stand-ins
for plans (no GPU)."""
import pytest

torch = pytest.importorskip("torch")

import outlier_split_mixed_b200 as osm  # noqa: E402


@pytest.mark.parametrize("epi", [osm.EPI_GELU_BF16, osm.EPI_GELU_REQUANT, 9])
def test_a_quantised_layer_refuses_an_activation_before_the_residual(epi):
    # it would be left out: the product onto a residual stream has none
    lin = object.__new__(osm.QuantLinear)
    x, r = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(4, 64)
    with pytest.raises(ValueError, match="GELU"):
        lin.forward(x, epi=epi, residual=r)
    with pytest.raises(ValueError, match="residual"):
        lin.forward(x, epi=epi, gate=r)
