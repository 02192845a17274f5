"""The training example: top-K extraction, distillation in place and sampling together."""
import pytest
import torch

import dflash2_draft_head_gb300 as df2
from dflash2_draft_head_gb300 import train_draft

pytestmark = pytest.mark.gpu


def test_training_lowers_the_loss_and_raises_acceptance():
    df2.build_library()
    r = train_draft.train(steps=60)
    torch.cuda.synchronize()
    assert df2.take_device_faults() == 0
    assert r["loss"][1] < 0.5 * r["loss"][0]
    assert r["accepted"][1] > r["accepted"][0] + 0.2


def test_a_run_can_be_repeated():
    a, b = (train_draft.train(steps=3, blocks=4) for _ in range(2))
    assert a == b
