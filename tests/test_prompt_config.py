"""Host-side checks of the operators that take a prompt through the block,
which return before any device work (no GPU): argument rules, null handles, the
packed argument structs against the header's layout, and the benchmark cases'
plain description."""

import ctypes
import importlib.util
import os
import random
import re
import shutil
import struct
import subprocess

import pytest

pytest.importorskip("torch")

from calibration_free_sparse_gb300 import block as BK
from calibration_free_sparse_gb300 import build as B
from calibration_free_sparse_gb300 import experts as EX
from calibration_free_sparse_gb300 import reader as RD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 256 * 1024   # aligned addresses that are never dereferenced


@pytest.fixture(scope="module")
def lib():
    B.build()
    return RD.library()


def test_null_handles(lib):
    for name in ("kv_chunk", "kv_collect", "kv_compact", "kv_fork", "kv_copy", "experts_activate",
                 "experts_combine"):
        fn = getattr(lib, "moe_reader_" + name)
        assert fn(None, b"\0" * 256, None) == RD.EINVAL
        assert fn(None, None, None) == RD.EINVAL
    assert lib.moe_reader_experts_plan(None, None) == RD.EINVAL
    assert lib.moe_reader_experts_status(None, None) == RD.EINVAL
    lib.moe_reader_experts_destroy(None)


GOOD = dict(hidden=256, inter=128, num_experts=8, type=1, flags=0)


def create(lib, gate=FAKE, up=2 * FAKE, down=3 * FAKE, **over):
    cfg = EX.Config(*dict(GOOD, **over).values())
    out = ctypes.c_void_p(123)
    code = lib.moe_reader_experts_create(ctypes.byref(cfg), gate, up, down, None, ctypes.byref(out))
    assert out.value is None
    return code


@pytest.mark.parametrize("over", [
    dict(hidden=0), dict(hidden=12), dict(hidden=65544), dict(inter=0), dict(inter=100),
    dict(inter=65544), dict(num_experts=0), dict(num_experts=1025), dict(type=0), dict(type=3),
    dict(flags=1), dict(gate=None), dict(up=None), dict(gate=None, up=None, down=None),
    dict(gate=FAKE + 8), dict(up=FAKE + 2), dict(down=FAKE + 4)])
def test_experts_configuration_rules(lib, over):
    assert create(lib, **over) == RD.EINVAL


def test_experts_report_a_failed_allocation(lib):
    assert lib.moe_reader_inject_fault(None, RD.INJECT_ALLOC_FAIL) == RD.OK
    assert create(lib) == RD.ENOMEM


PLAN = ("ids", "order", "offsets", "places", "skipped", "tokens", "topk", "experts")


@pytest.mark.parametrize("over", [
    dict(ids=0), dict(order=0), dict(offsets=0), dict(places=0), dict(skipped=0), dict(tokens=-1),
    dict(topk=0), dict(topk=65), dict(experts=0), dict(experts=1025), dict(ids=FAKE + 2),
    dict(order=FAKE), dict(places=2 * FAKE), dict(offsets=2 * FAKE + 60), dict(skipped=4 * FAKE + 8),
    dict(tokens=1 << 29, topk=2)])
def test_experts_plan_rules(lib, over):
    a = dict(ids=FAKE, order=2 * FAKE, offsets=3 * FAKE, places=4 * FAKE, skipped=5 * FAKE, tokens=8,
             topk=2, experts=8)
    a.update(over)
    assert lib.moe_reader_experts_plan(EX._PLAN.pack(*(a[n] for n in PLAN)), None) == RD.EINVAL


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs a C compiler")
def test_packed_structs_match_the_header(tmp_path):
    """Sizes and every field's offset of the argument structs."""
    text = open(os.path.join(ROOT, "include", "moe_reader.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    formats = {"kv_chunk": BK._CHUNK, "kv_pages": BK._PAGES, "kv_fork": BK._FORK,
               "kv_copy": BK._COPY, "experts_plan": EX._PLAN, "experts_activate": EX._ACTIVATE,
               "experts_combine": EX._COMBINE}
    lines, want = [], []
    for name, fmt in formats.items():
        body = re.search(r"typedef struct \{([^}]*)\} moe_reader_%s_args;" % name, text).group(1)
        fields = [f.strip().split()[-1].strip("* ") for decl in body.split(";") if decl.strip()
                  for f in decl.split(",")]
        kinds = "".join(k * int(n or 1) for n, k in re.findall(r"(\d*)([a-z])",
                                                             fmt.format.replace("4x", ""), re.I))
        assert len(kinds) == len(fields), name
        at = 0
        for f, k in zip(fields, kinds):
            lines.append(f'printf("%zu\\n", offsetof(moe_reader_{name}_args, {f}));')
            want.append(at)
            at += struct.calcsize(k)
        lines.append(f'printf("%zu\\n", sizeof(moe_reader_{name}_args));')
        want.append(fmt.size)
    cfg = dict(hidden=0, inter=4, num_experts=8, type=12, flags=16)
    for f, at in cfg.items():
        lines.append(f'printf("%zu\\n", offsetof(moe_reader_experts_config, {f}));')
        want.append(at)
    src = tmp_path / "sizes.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"moe_reader.h\"\n"
                   "int main(void) {\n" + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(g) for g in got] == want


def test_operator_cases_are_consistent():
    """The benchmark cases' plain description: names, work and lengths."""
    spec = importlib.util.spec_from_file_location(
        "more_operator_cases", os.path.join(ROOT, "perf", "more_operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    cases = m.listed()
    assert len({c["name"] for c in cases}) == len(cases) <= 12
    rng = random.Random(4)
    for c in cases + [m.draw(rng) for _ in range(50)]:
        w = m.work(c)
        assert w["bytes"] > 0 and w["flops"] > 0
