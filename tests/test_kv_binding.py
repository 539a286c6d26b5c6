"""What the binding makes of arguments before the library sees them (no GPU needed but for one)."""
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402


def test_rope_table_from_a_parameter():
    """A model's own frequencies: a parameter that wants gradients."""
    freq = torch.nn.Parameter(torch.tensor([1.0, 0.25]))
    t = q.rope_table(5, 4, inv_freq=freq, device="cpu")
    assert not t.requires_grad and torch.equal(t, q.rope_table(5, 4, inv_freq=[1.0, 0.25], device="cpu"))


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
def test_rope_table_from_frequencies_on_the_gpu():
    t = q.rope_table(5, 4, inv_freq=torch.tensor([1.0, 0.25], device="cuda"))
    assert torch.equal(t.cpu(), q.rope_table(5, 4, inv_freq=[1.0, 0.25], device="cpu"))
