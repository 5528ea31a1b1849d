"""The library's choices by sizes (csrc/rules.h), compiled for the host: which form of the product
a call takes, and how the balance loss cuts its tokens."""

import ctypes
import functools
import os
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FORMS = ("large", "128x128", "128x128 deep", "64x128", "128x64", "64x64", "64x32 deep", "64x32",
         "32x32", "32x16", "16x16")

SOURCE = """
#include "rules.h"
static_assert(uep::kPrForms == %d, "the forms' names");
extern "C" {
int form(int64_t rows, int n_inst, int n_out, int D, int glu) {
  return uep::pr_form(rows, n_inst, n_out, D, glu != 0);
}
int lanes(int E, int size) { return uep::bl_lanes_of(E, size); }
int chunk(int64_t n_tok, int E, int size, int grad) {
  return uep::bl_chunk_tokens(n_tok, E, size,
                              grad ? uep::kBlGradBlocks : uep::bl_sum_blocks(n_tok, E, size));
}
int sliced(int64_t mean, int E) { return uep::bl_sliced(mean, E); }
int threads() { return uep::kBlThreads; }
}
""" % len(FORMS)


@functools.lru_cache(maxsize=None)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "rules.cc"), os.path.join(d, "rules.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        try:
            subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                            os.path.join(ROOT, "moe_expert_load_amd", "csrc"), src, "-o", lib],
                           check=True, capture_output=True, text=True)
        except FileNotFoundError:
            pytest.skip("no g++")
        return ctypes.CDLL(lib)


def form(rows, n_inst, n_out, D, glu):
    return FORMS[_lib().form(ctypes.c_int64(rows), n_inst, n_out, D, int(glu))]


def chunk(n_tok, E, size, grad=False):
    """Tokens of a chunk, and how many passes a block makes over them."""
    n = _lib().chunk(ctypes.c_int64(n_tok), E, size, int(grad))
    return n, n * _lib().lanes(E, size) // _lib().threads()


def sliced(mean, E):
    """Whether several blocks join a sequence of so many chunks on the average."""
    return bool(_lib().sliced(ctypes.c_int64(mean), E))
