"""The limits in projection.py are those of include/moe_proj.h."""
import os
import re

import pytest

from routed_expert_mlp_amd import projection as P

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_proj.h")


@pytest.mark.parametrize("name", ["NORM_MAX_HIDDEN", "LORA_MAX_RANK", "MAX_FEATURES"])
def test_limits(name):
    value = re.search(rf"#define MOE_PROJ_{name}\s+\(?([0-9 <]+)\)?", open(HEADER).read()).group(1)
    base, _, shift = value.partition("<<")
    assert getattr(P, name) == int(base) << int(shift or 0)
