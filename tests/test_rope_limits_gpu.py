"""Rotary positions and linear attention at the ends of what the sizes' integers hold."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_recurrence_11_b200 import kda
    return kda


@pytest.mark.parametrize("shape", [(1, (1 << 32) + 3, 1, 2), ((1 << 32) + 3, 1, 1, 2)])
def test_more_tokens_than_an_integer_counts(K, shape):
    """Refused, and not taken for the three tokens that 32 bits of their number say."""
    q = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(K.KdaError) as e:
        K.kda_rope(q, None, torch.ones(1, device="cuda"), q_out=q)
    assert e.value.code == K.KDA_ERR_UNSUPPORTED


def test_more_heads_or_channels_than_an_integer_counts(K):
    inv = torch.ones(1, device="cuda")
    for shape in ((1, 1, (1 << 32) + 1, 2), (1, 1, 1, (1 << 32) + 2)):
        q = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(K.KdaError) as e:
            K.kda_rope(q, None, inv, q_out=q)
        assert e.value.code == K.KDA_ERR_UNSUPPORTED
    q = torch.empty(1, 1, 1, (1 << 32) + 32, dtype=torch.bfloat16, device="cuda")
    v, g = torch.empty(1, 1, 1, 32, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, device="cuda")
    for f in (lambda: K.kda_hla_forward(q, q, v, g, return_state=False), lambda: K.kda_hla_backward(q, q, v, g, v, return_dS0=False)):
        with pytest.raises(K.KdaError) as e:
            f()
        assert e.value.code == K.KDA_ERR_UNSUPPORTED
