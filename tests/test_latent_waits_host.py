"""Waits between the roles of the latent attention's kernels, as their sources have them."""
import os
import re

import pytest

from hybrid_linear_attention_conv_gb300 import build as gbuild


@pytest.mark.parametrize("name", ["gdn_latent_tiles.cu", "gdn_latent_expanded.cu"])
def test_no_role_arrives_at_a_hardware_barrier_that_another_waits_at(name):
    """A hardware barrier counts arrivals and not who they are: a role that arrives without waiting may come twice after a
    wait that gave up, completes the barrier by itself, and leaves the role that waits there without an end."""
    with open(os.path.join(gbuild.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert "named_sync" in text
    assert not re.search(r"named_arrive|bar\.arrive|barrier\.arrive", text)
