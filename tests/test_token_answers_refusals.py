"""What AnswerHead.answer refuses before it runs anything."""
import pytest
import torch

from conv_bn_silu_gb300.token_head import AnswerHead


@pytest.mark.parametrize("shape", [(1,), (2, 2), (6, 1, 2)])
def test_first_tokens_of_another_number(shape):
    """One would be every answer's, silently."""
    head = object.__new__(AnswerHead)
    head.images, head.answers, head.max_answer, head.graph = 2, 3, 8, None
    head.start = lambda cells: pytest.fail("started")
    with pytest.raises(ValueError, match="first tokens"):
        head.answer(torch.zeros(2, 4), torch.zeros(shape, dtype=torch.int64), 4)
