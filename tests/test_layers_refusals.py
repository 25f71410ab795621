"""The refusals of test_layers_host.py for what is wrong with them: a machine without a GPU
answers Z1_EINVAL to any call that gets as far as its stream, so here a pointer that is not
in question is misaligned too, and a call that is not refused for its values ends with
Z1_EALIGN."""
import pytest

import test_layers_host as H
from mixed_precision_zero_amd import binding as B
from test_layers_alias import status


def listed(test):
    """The values of `over` of a test that are refused with Z1_EINVAL."""
    for mark in test.pytestmark:
        if mark.args[0].startswith("over"):
            return [o if isinstance(o, dict) else o[0] for o in mark.args[1] if isinstance(o, dict) or o[1] == B.Z1_EINVAL]
    raise LookupError(test)


def cases():
    for call, tests in (("z1_dropout", [H.test_dropout_refuses]),
                        ("z1_linear", [H.test_linear_refuses, H.test_linear_refuses_outputs_over_other_buffers]),
                        ("z1_linear_dz", [H.test_linear_dz_refuses]),
                        ("z1_linear_grad", [H.test_linear_grad_refuses, H.test_linear_grad_refuses_outputs_over_other_buffers]),
                        ("z1_qk_norm_rope", [H.test_qk_refuses]), ("z1_qk_norm_rope_grad", [H.test_qk_refuses])):
        for test in tests:
            for over in listed(test):
                yield call, over
    overlaps = [dict(q_out=0x100000, q_out_token=512), dict(q_out=0x100000, q_out_head=128), dict(q_out=0x210000), dict(q_out=0x200000)]
    for over in overlaps:
        yield "z1_qk_norm_rope", over
    for over in overlaps + [dict(q_out=0x120000, q_out_token=512), dict(q_out=0x220000), dict(q_dweight=0x240000), dict(q_dout=None),
                            dict(q_weight=None)]:
        yield "z1_qk_norm_rope_grad", over


@pytest.mark.parametrize("call,over", list(cases()))
def test_refused_for_its_values(call, over):
    assert status(call, over) == B.Z1_EINVAL
