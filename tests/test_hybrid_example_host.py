"""The hybrid example's own checks, on the CPU with a stack that does nothing."""
import pytest
import torch

from gated_delta_rule_44_gb300 import hybrid_example as E


class Doubles:
    def step(self, x, lens, kv_lens, new):
        assert x.shape[0] == sum(lens)
        return 2 * x


def test_every_row_comes_from_its_own_sequence():
    x = torch.arange(14.0)[:, None].repeat(1, 3)
    out = E.generate(Doubles(), x, [4, 1, 3], [6, 3, 5])
    assert torch.equal(out, 2 * x)


@pytest.mark.parametrize("prompts,totals,rows", [
    ([3, 2], [5, 7], 12),       # 2 and 5 further tokens
    ([2, 3], [7, 5], 12),
    ([3, 2], [2, 1], 3),        # fewer tokens than the prompts
    ([3, 2], [5, 4], 10),       # more rows than tokens
    ([3], [5, 2], 7),           # a sequence without a prompt
])
def test_unequal_numbers_of_further_tokens_are_refused(prompts, totals, rows):
    with pytest.raises(ValueError):
        E.generate(Doubles(), torch.ones(rows, 3), prompts, totals)
