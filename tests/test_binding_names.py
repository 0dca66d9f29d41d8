"""Every bound function under the names that the documentation gives it: an attribute of the
package and of `kda`."""
import inspect

import pytest

import gated_delta_rule_57_gb300 as pkg
from gated_delta_rule_57_gb300 import kda, latent

BOUND = sorted(n for n in set(kda.header_functions()) | set(pkg.__all__) if hasattr(pkg, n))


def test_the_header_is_bound():
    assert {"kda_chunk_fwd", "kda_attn_paged", "kda_kv_append_rope", "kda_latent_append", "kda_attn_latent_prompt",
            "kda_attn_latent_paged", "kda_attn_latent_workspace_size", "kda_rope_turns"} <= set(BOUND)


@pytest.mark.parametrize("name", BOUND)
def test_is_the_same_under_every_name(name):
    assert getattr(kda, name) is getattr(pkg, name)
    if hasattr(latent, name):
        assert getattr(latent, name) is getattr(pkg, name)


def test_latent_functions_by_import_and_listing():
    from gated_delta_rule_57_gb300.kda import kda_attn_latent_paged
    assert kda_attn_latent_paged is latent.kda_attn_latent_paged
    defined = {n for n, f in vars(latent).items() if n.startswith("kda_") and inspect.isfunction(f)}
    assert defined <= set(dir(kda)) and defined <= set(pkg.__all__)


def test_other_names_are_refused():
    with pytest.raises(AttributeError, match="kda_nothing"):
        kda.kda_nothing
