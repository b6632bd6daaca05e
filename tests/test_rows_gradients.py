"""Operators on logits rows that form no gradient refuse tensors that want
one (no GPU: the refusal comes before anything else is looked at)."""

import pytest
import torch
from torch.autograd import forward_ad

import speculative_decoding_verification_46_gb300 as sv


def _grad(*shape):
    return torch.zeros(*shape, requires_grad=True)


ROWS = torch.zeros(2, 3, 16)
IDX, LP = torch.zeros(2, 3, 4, dtype=torch.int32), torch.zeros(2, 3, 4)
HIST, LEN = torch.zeros(2, 5, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)


@pytest.mark.parametrize("name, call", [
    ("logits", lambda: sv.adjust_logits(_grad(2, 3, 16))),
    ("logits", lambda: sv.adjust_logits(_grad(2, 3, 16) * 2)),
    ("repetition", lambda: sv.adjust_logits(ROWS, history=HIST, history_len=LEN, repetition=_grad(2))),
    ("frequency", lambda: sv.adjust_logits(ROWS, history=HIST, history_len=LEN, frequency=_grad(2))),
    ("presence", lambda: sv.adjust_logits(ROWS, history=HIST, history_len=LEN, presence=_grad(2))),
    ("bias_values", lambda: sv.adjust_logits(ROWS, bias_tokens=IDX[0], bias_values=_grad(3, 4))),
    ("out", lambda: sv.adjust_logits(ROWS, out=_grad(2, 3, 16))),
    ("out", lambda: sv.adjust_logits(ROWS, out=_grad(2, 3, 16) + 1)),
    ("logits", lambda: sv.top_logits(_grad(2, 3, 16), 4)),
    ("logprobs", lambda: sv.top_logits(ROWS, 4, outputs=(IDX, _grad(2, 3, 4), torch.zeros(2, 3)))),
    ("tail", lambda: sv.top_logits(ROWS, 4, outputs=(IDX, LP, _grad(2, 3)))),
    ("out_grad", lambda: sv.distill_loss_grad(ROWS, IDX, LP, out_grad=_grad(2, 3, 16))),
    ("weight", lambda: sv.distill_loss_grad(ROWS, IDX, LP, weight=_grad(2, 3))),
])
def test_refuses_what_wants_a_gradient(name, call):
    with pytest.raises(ValueError, match=f"no gradient is formed for {name}"):
        call()
    # nobody asks for one there: the next check is that the tensors are CUDA ones
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        call()


def test_the_gradient_may_take_the_place_of_a_student_that_requires_one():
    """Documented: nothing is recorded, and the caller hands the gradient on."""
    for student in (_grad(2, 3, 16), _grad(2, 3, 16) * 2):
        with pytest.raises(ValueError, match="CUDA"):
            sv.distill_loss_grad(student, IDX, LP, out_grad=student)


def test_refuses_forward_mode():
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(torch.zeros(2, 3, 16), torch.ones(2, 3, 16))
        student = forward_ad.make_dual(torch.zeros(2, 3, 16, requires_grad=True), torch.ones(2, 3, 16))
        for call in (lambda: sv.adjust_logits(dual), lambda: sv.top_logits(dual, 4), lambda: sv.distill_loss_grad(dual, IDX, LP),
                     lambda: sv.distill_loss_grad(student, IDX, LP)):
            with pytest.raises(ValueError, match="no gradient is formed for"):
                call()
        with pytest.raises(ValueError, match="CUDA"):
            sv.adjust_logits(ROWS)
