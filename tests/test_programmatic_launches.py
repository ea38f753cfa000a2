"""Kernels launched with programmatic stream serialisation start while earlier kernels of the stream
may still write, so behind their wait they load coherently. A read of the CUDA sources, on the CPU:
whether a read-only load returns an old value depends on the compiler and on what a cache holds."""
import os
import re

import pytest

from fp32_accumulate_lm_b200 import _build

WAIT = "pdl_wait()"
# (and the intrinsics with a cache hint, which the compiler need not keep behind the wait)
READ_ONLY = re.compile(r"__ld(g|cs|cg|ca|lu)\s*\(|__restrict__|\bld\.global\.(\w+\.)*nc\b")


def source(name):
    """A source file without its comments."""
    text = open(os.path.join(_build.CSRC, name)).read()
    return re.sub(r"/\*.*?\*/", "", re.sub(r"//[^\n]*", "", text), flags=re.S)


def functions(text):
    """(signature, body) of every device function and kernel."""
    for m in re.finditer(r"\b(__global__|__device__)\b", text):
        opened = text.find("{", m.start())
        ended = text.find(";", m.start())
        if opened < 0 or 0 <= ended < opened:
            continue
        depth, at = 0, opened
        while True:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
            if depth == 0:
                break
        yield m.group(1), text[m.start():opened], text[opened:at]


def kernels(name):
    return [(head, body) for kind, head, body in functions(source(name)) if kind == "__global__"]


FILES = sorted(os.path.basename(p) for p in _build.sources() if p.endswith((".cu", ".cuh")))


def launched_programmatically():
    """The names of the kernels that launch_head is given, directly or through a choice."""
    host = source("lmhead.cu") + source("lmhead_train_entry.cuh")
    found = set()
    for m in re.finditer(r"launch_head\(", host):
        found |= set(re.findall(r"lmh::(\w+_kernel)", host[m.end():m.end() + 400].split(";")[0]))
    for name in re.findall(r"auto (?:fold|kernel) =([^;]*);", host):
        found |= set(re.findall(r"lmh::(\w+_kernel)", name))
    return found


def test_the_reader_of_sources_finds_the_kernels():
    names = launched_programmatically()
    assert {"xent_gemm_kernel", "xent_pack_kernel", "xent_fold_kernel", "xent_reduce_kernel",
            "xent_rows_kernel", "xent_bias_kernel", "xent_finish_kernel", "embed_kernel",
            "embed_sort_kernel", "embed_sum_kernel", "embed_join_kernel"} <= names
    assert READ_ONLY.search("__ldg(p + 1)") and READ_ONLY.search("const int* __restrict__ p")
    assert READ_ONLY.search("ld.global.nc.v4.f32") and READ_ONLY.search("__ldcs(p)")
    assert not READ_ONLY.search("ld.global.cs.v4.f32") and not READ_ONLY.search("load_cs(p)")


@pytest.mark.parametrize("name", FILES)
def test_kernels_that_wait_load_coherently(name):
    for head, body in kernels(name):
        if WAIT in body:
            assert not READ_ONLY.search(head + body), head


@pytest.mark.parametrize("name", ["lmhead_xent.cuh", "lmhead_embed.cuh"])
def test_what_those_kernels_call_loads_coherently(name):
    """Every kernel of these files is launched so, and their functions are called by nothing else."""
    for head, body in kernels(name):
        assert WAIT in body, head
    for _, head, body in functions(source(name)):
        assert not READ_ONLY.search(head + body), head


def test_every_kernel_launched_so_waits():
    names = launched_programmatically()
    for name in FILES:
        for head, body in kernels(name):
            kernel = re.search(r"(\w+_kernel)\s*\(", head).group(1)
            assert kernel not in names or WAIT in body, kernel
