"""Which problem structures the compiled binding takes, told on the CPU: the problem is looked at before the tensors."""
import pytest
import torch

import dispatch_fp8_grouped_topk_amd as mm

PROBLEMS = dict(norm=mm.NormProblem.make(4, 256), gate=mm.GateProblem.make(4, 256, 8), topk=mm.TopkProblem.make(4, 8, 2),
                sort=mm.SortProblem.make(4, 256, 8, 2), unsort=mm.UnsortProblem.make(4, 256, 2),
                product=mm.ProductProblem.make(4, 256, 256), act=mm.ActProblem.make(4, 256))
CALLS = dict(norm=[(mm.mega_moe_norm_quant, 2)], gate=[(mm.mega_moe_gate_logits, 3)], topk=[(mm.mega_moe_gate_topk, 3)],
             sort=[(mm.mega_moe_sort_tokens, 6)], unsort=[(mm.mega_moe_unsort_tokens, 3), (mm.mega_moe_unsort_backward, 2)],
             product=[(mm.mega_moe_block_product, 5)], act=[(mm.mega_moe_act_quant, 1), (mm.mega_moe_act_backward, 3)])


@pytest.mark.parametrize("op", CALLS)
@pytest.mark.parametrize("other", PROBLEMS)
def test_every_operator_takes_its_own_problem_only(op, other):
    """Structures of the same size are told apart; what is wrong with the tensors comes after."""
    host = torch.zeros(4, 256)
    for call, tensors in CALLS[op]:
        with pytest.raises(ValueError, match="device tensors" if other == op else "problem must be"):
            call(PROBLEMS[other], *[host] * tensors)
    with pytest.raises(ValueError, match="problem must be"):
        CALLS[op][0][0](b"\0" * 40, *[host] * CALLS[op][0][1])


def test_a_subclass_of_a_problem_is_one():
    class Mine(mm.SortProblem):
        pass

    with pytest.raises(ValueError, match="device tensors"):
        mm.mega_moe_sort_tokens(Mine.make(4, 256, 8, 2), *[torch.zeros(4, 256)] * 6)
