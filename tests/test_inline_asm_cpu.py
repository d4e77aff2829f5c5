"""Inline assembly in the kernels names the registers that it writes beside its
operands: the compiler may hold a value of its own in them."""

import glob
import os
import re

import combine_expert_ffn_amd as M

CSRC = os.path.join(os.path.dirname(M.__file__), "csrc")


def _statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        text = open(path).read()
        for m in re.finditer(r"\basm\s*(?:volatile\s*)?\(", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[i], 0)
                i += 1
            yield os.path.basename(path), text[m.end(): i - 1]


def test_m0_is_a_clobber_where_it_is_written():
    writes = [(f, s) for f, s in _statements() if re.search(r"\bs_\w+ m0\b", s)]
    assert writes
    for f, s in writes:
        clobbers = s.split(":")[-1]
        assert '"m0"' in clobbers, (f, s)
