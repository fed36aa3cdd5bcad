"""The latent-attention sources hold no function that nothing calls."""
from __future__ import annotations

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "kimi_delta_attention_19_b200", "csrc")


def test_every_function_is_called():
    text = ""
    for name in glob.glob(os.path.join(CSRC, "kda_latent*")):
        with open(name) as f:
            text += re.sub(r"//.*", "", f.read())
    defined = set(re.findall(r"\b(\w+)\s*\([^;{}]*\)\s*\{", text)) - {"switch", "if", "for", "while"}
    assert len(defined) > 50
    idle = {n for n in defined if len(re.findall(rf"\b{n}\b", text)) == 1}
    assert {n for n in idle if not n.startswith("kda_latent_")} == set()     # (those are the ABI)
