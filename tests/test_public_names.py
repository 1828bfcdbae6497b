"""What `from kda_recurrent_state_amd import *` gives: every part's public functions (CPU)."""
import pytest

import kda_recurrent_state_amd as kda
from kda_recurrent_state_amd import block, feedforward, state_cache, statespace


@pytest.mark.parametrize("part", [block, statespace, feedforward, state_cache], ids=lambda m: m.__name__.split(".")[-1])
def test_names_of_a_part(part):
    given = {}
    exec("from kda_recurrent_state_amd import *", given)
    for name in part.__all__:
        assert name in kda.__all__ and given[name] is getattr(part, name) is getattr(kda, name), name


def test_each_name_once():
    assert len(set(kda.__all__)) == len(kda.__all__)
