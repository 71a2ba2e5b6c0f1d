"""The generation example's checks, without a GPU."""
import importlib.util
import os
import types

import pytest

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "generate.py")


@pytest.mark.parametrize("prompts", [[[1, 2], []], [[], [1]], [[1]], [[1], [2], [3]], []])
def test_prompts_that_do_not_fit_the_server_are_refused(prompts):
    spec = importlib.util.spec_from_file_location("generate_example_host", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # an empty prompt has no last row: the row before it, of another request, would be taken for it
    with pytest.raises(ValueError, match="prompts of one token or more"):
        example.generate(types.SimpleNamespace(R=2), prompts, 3)
