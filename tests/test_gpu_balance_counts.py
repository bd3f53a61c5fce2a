"""Counts of the balance loss above 2^31: given experts may name one expert in
several slots of a row, so a count can reach T top_k."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_count_above_32_bits():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    T, E, k = (1 << 26) + 3, 32, 32
    if torch.cuda.mem_get_info()[0] < 26 << 30:
        pytest.skip("needs 26 GB of GPU memory")
    from entropy_loss_gb300 import build, flp
    build.build()
    z = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    experts = torch.full((T, k), 5, device="cuda")
    experts[:2, 0] = 7
    loss, _, counts = flp.balance_loss(z, k, experts=experts, grad=False)
    assert counts[5] == T * k - 2 > 1 << 31 and counts[7] == 2 and counts.sum() == T * k
    assert abs(float(loss) - 1) <= 2.0 ** -17 * (1 + (E - 1) / E + (E - 1) / E)   # even probabilities
