"""Kernels that are launched while the kernel before them may still run must not read what that
one writes until they have waited for it, and not by read-only loads at all: those ask that
nothing writes during the kernel's life.  Whether a GPU run meets a violation is chance, so the
sources of the packed operators and of the many-tensor AdamW are checked."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "layer_streamed_qlora_nf4_b200", "csrc")
FILES = ["packed.cu", "packed_attention.cu", "adamw_multi.cu"]


def _bare(text):
    """Without comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def _block(text, at, pair="{}"):
    """The bracketed text that starts at or behind `at`, and its end."""
    a = text.index(pair[0], at)
    depth = 0
    for i in range(a, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return text[a:i + 1], i + 1
    raise AssertionError("unbalanced")


def kernels(text):
    """-> (name, parameters, body) of every __global__ function."""
    text = _bare(text)
    for m in re.finditer(r"__global__", text):
        at = m.end()
        b = re.compile(r"\s*(void)?\s*__launch_bounds__").match(text, at)
        if b:
            at = _block(text, b.end(), "()")[1]
        n = re.compile(r"\s*(?:void\s+)?(\w+)\s*\(").match(text, at)
        params, end = _block(text, n.end() - 1, "()")
        yield n.group(1), params, _block(text, end)[0]


def early_reads(params, body):
    """Reads through pointer parameters, or members of an index, before the wait."""
    head = body[:body.index("pdl_wait();")]
    names = re.findall(r"\*\s*(?:const\s+)?(\w+)\s*[,)]", params)
    bad = [n for n in names if re.search(r"\b%s\s*\[|[^\w)\s]\s*\*\s*%s\b" % (n, n), head)]
    for n in re.findall(r"PackedIndex\s+(\w+)", params):
        bad += re.findall(r"\b%s\.\w+" % n, head)
    return bad


@pytest.mark.parametrize("name", FILES)
def test_nothing_is_read_before_the_wait_or_by_read_only_loads(name):
    text = open(os.path.join(CSRC, name)).read()
    found = 0
    for kernel, params, body in kernels(text):
        if "pdl_wait();" not in body:
            continue
        found += 1
        assert "__restrict__" not in params, kernel   # (such const data are read that way)
        assert not early_reads(params, body), (kernel, early_reads(params, body))
    assert found >= 3
    assert not re.search(r"__ldg\b|ld\.global\.nc|__restrict__", _bare(text))


def test_the_check_sees_an_early_read():
    src = """template <int D>
    __global__ void __launch_bounds__(640, 1)
        k(PackedIndex idx, const float* a, int n, int* taken) { // a[0]
      %s
      pdl_wait();
      const float y = a[1] + idx.head[0];
    }"""
    for early, bad in (("const float* x = a + n;", []), ("float x = a[n];", ["a"]),
                       ("int x = n + *taken;", ["taken"]), ("int x = idx.head[0];", ["idx.head"]),
                       ("const int x = idx.pos[n]; // nothing", ["idx.pos"])):
        (name, params, body), = kernels(src % early)
        assert name == "k" and early_reads(params, body) == bad, early


def test_the_attention_of_equal_sequences_too():
    text = open(os.path.join(CSRC, "attention.cu")).read()
    found = [k for k, params, body in kernels(text) if "pdl_wait();" in body and
             "__restrict__" not in params and not early_reads(params, body)]
    assert len(found) == 3 and not re.search(r"__ldg\b|ld\.global\.nc", _bare(text))
