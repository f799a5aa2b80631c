"""A profile read returns every kernel that the library names, however many ran."""

import os
import re

from gated_delta_rule_54_amd import binding

CSRC = os.path.join(os.path.dirname(binding.__file__), "csrc")


def names():
    found = set()
    for f in sorted(os.listdir(CSRC)):
        for line in open(os.path.join(CSRC, f)):
            if re.search(r"\bProfScope \w+\(", line):
                found |= set(re.findall(r'"(\w+)"', line))
    return sorted(found)


def test_a_read_of_all_kernels(monkeypatch):
    all_names = names()
    assert {"seq_fwd", "chunk_grad", "linear_token", "norm_bwd", "rotary", "cache_append", "attention_join"} <= set(all_names)

    class Lib:
        @staticmethod
        def gdr_profile_read(buf, cap, n):
            for i, name in enumerate(all_names[:cap]):
                buf[i] = binding.GdrKernelTime(name.encode(), float(i), i + 1)
            n._obj.value = len(all_names)
            return binding.GDR_OK

    monkeypatch.setattr(binding, "lib", lambda: Lib)
    got = binding.gdr_profile_read()
    assert got == {name: (float(i), i + 1) for i, name in enumerate(all_names)}
