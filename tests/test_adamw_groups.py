"""A group of AdamW takes lr and weight_decay; what it cannot take is refused, not ignored."""
import pytest
import torch

from hybrid_upcycling_gb300 import AdamW


@pytest.mark.parametrize("extra", [{"betas": (0.5, 0.9)}, {"eps": 1e-3}, {"wd": 0.0}, {"max_norm": 1.0}])
def test_other_settings_of_a_group_are_refused(extra):
    p, q = torch.zeros(3), torch.zeros(4)
    with pytest.raises(ValueError, match=next(iter(extra))):
        AdamW([{"params": [p]}, {"params": [q], "lr": 0.1, **extra}])


def test_its_own_settings_are_kept():
    opt = AdamW([{"params": [torch.zeros(3)], "weight_decay": 0.0}, {"params": iter([torch.zeros(4)]), "lr": 0.1}], lr=0.2,
                weight_decay=0.3)
    assert [(g["lr"], g["weight_decay"], len(g["params"])) for g in opt.groups] == [(0.2, 0.0, 1), (0.1, 0.3, 1)]
