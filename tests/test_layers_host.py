"""The layers between convolutions, checked on the CPU: what their sources may hold, and
the arithmetic of their kernels that runs as plain host code."""

import glob
import os

import pytest

from sparse_convolution_hash_gb300 import build as libbuild


def test_no_load_fills_several_ctas():
    """The library runs on every GPU of a job: a bulk load goes to its own CTA only.  (A commit of the
    tensor core may arrive on both barriers of a CTA pair: it moves no data.)"""
    sources = [f for d in (libbuild.CSRC, libbuild.CSRC_LAYERS) for f in glob.glob(os.path.join(d, "*"))]
    assert sources
    for f in sources:
        with open(f, encoding="utf-8") as fh:
            text = fh.read()
        for piece in text.split("cp.async.bulk")[1:]:
            assert "multi" + "cast" not in piece.split('"')[0], f
