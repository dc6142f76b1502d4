"""What the library's translation units share is used: every function of attn_host.h has a caller."""
import os
import re

from attention_forward_tiled_b200 import build as abuild


def test_shared_functions_have_callers():
    def read(name):
        with open(os.path.join(abuild.CSRC, name)) as f:
            return f.read()

    header = read("attn_host.h")
    names = set(re.findall(r"\b(\w+)\([^;{}]*\)\s*[;{]", re.sub(r"//.*", "", header)))
    names = {n for n in names if re.search(rf"^(inline |template.*\n)?[\w ]+ {n}\(", header, re.M)}
    assert {"host_device", "host_encode_bnhd", "cuda_failed"} <= names
    users = read("attn_window.cu") + header
    for n in names:
        assert len(re.findall(rf"\b{n}\b", users)) >= 2, n  # its declaration and a use
