"""The example block: latent attention and the MoE layer, a prompt then single tokens.

Both ways round the same values to bf16 (u = 2^-8) at keys, values, weights, latent queries and outputs and at the two
outer products, about eight roundings on the path, and the MoE layer quantises its input to 8 bits (half a step, 2^-8 of
a block's largest): 9 * 2^-8 = 3.5e-2 bounds their sum.  A token attended wrongly is off by tenths."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("args", [["--prompt", "200", "--steps", "5"], ["--prompt", "33", "--steps", "3", "--fp8"]])
def test_block(args):
    spec = importlib.util.spec_from_file_location("latent_block", os.path.join(ROOT, "examples", "latent_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    print("latent block", args, flush=True)
    assert m.main(args) < 3.5e-2
