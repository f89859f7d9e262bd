"""Host-side checks of the decode-step operators that return before any device
work (no GPU): the cache's configuration rules, null handles and arguments,
argument checks of the residual norm, and the packed argument structs against
the header's."""

import ctypes
import os
import re
import shutil
import struct
import subprocess

import pytest

from calibration_free_sparse_gb300 import block as BK
from calibration_free_sparse_gb300 import build as B
from calibration_free_sparse_gb300 import reader as RD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 256 * 1024   # aligned addresses that are never dereferenced
GOOD = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, num_pages=64,
            max_requests=4, cache_type=1, flags=0)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return RD.library()


def create(lib, k=FAKE, v=2 * FAKE, codes=None, steps=None, ks=None, vs=None, **over):
    cfg = BK.Config(*dict(GOOD, **over).values())
    out = ctypes.c_void_p(123)
    code = lib.moe_reader_kv_create(ctypes.byref(cfg), k, v, codes, steps, ks, vs, None,
                                    ctypes.byref(out))
    assert out.value is None
    return code


@pytest.mark.parametrize("over", [
    dict(num_q_heads=7), dict(num_q_heads=0), dict(num_q_heads=130), dict(num_kv_heads=0),
    dict(head_dim=96), dict(head_dim=32), dict(page_size=8), dict(page_size=48),
    dict(page_size=512), dict(num_pages=0), dict(num_pages=1 << 27), dict(max_requests=0),
    dict(max_requests=1025), dict(cache_type=0), dict(cache_type=4), dict(flags=1),
    dict(k=None), dict(v=None), dict(v=FAKE), dict(k=FAKE + 16), dict(v=FAKE * 2 + 128),
    dict(codes=FAKE), dict(steps=FAKE), dict(codes=FAKE + 8, steps=FAKE),
    dict(ks=FAKE), dict(ks=FAKE, vs=FAKE), dict(cache_type=3), dict(cache_type=3, ks=FAKE)])
def test_cache_configuration_rules(lib, over):
    assert create(lib, **over) == RD.EINVAL


def test_cache_reports_a_failed_allocation(lib):
    assert lib.moe_reader_inject_fault(None, RD.INJECT_ALLOC_FAIL) == RD.OK
    assert create(lib) == RD.ENOMEM


def test_null_handles(lib):
    for name in ("plan", "append", "attend", "select"):
        fn = getattr(lib, "moe_reader_kv_" + name)
        assert fn(None, b"\0" * 256, None) == RD.EINVAL
        assert fn(None, None, None) == RD.EINVAL
    assert lib.moe_reader_kv_status(None, None) == RD.EINVAL
    lib.moe_reader_kv_destroy(None)


NORM = ("h", "y", "gate", "post", "pre", "h_out", "x", "hs", "ys", "os", "xs", "grow", "gcol",
        "rows", "hidden", "ht", "yt", "xt", "gt", "wt", "scale", "eps")


@pytest.mark.parametrize("over", [
    dict(h=0), dict(x=0), dict(hidden=12), dict(hidden=0), dict(hidden=65544), dict(rows=-1),
    dict(ht=3), dict(yt=5), dict(xt=-1), dict(hs=252), dict(h=FAKE + 8), dict(pre=FAKE + 4),
    dict(post=FAKE * 9, y=0), dict(gate=FAKE * 9, y=0), dict(gate=FAKE * 9, gcol=2),
    dict(gate=FAKE * 9, gcol=1, grow=3), dict(gate=FAKE * 9 + 2), dict(x=FAKE), dict(x=2 * FAKE),
    dict(h_out=2 * FAKE), dict(h_out=FAKE + 1024, os=256), dict(h_out=FAKE, os=512),
    dict(pre=FAKE * 7, wt=3)])
def test_residual_norm_rules(lib, over):
    a = dict(h=FAKE, y=2 * FAKE, gate=0, post=0, pre=0, h_out=0, x=3 * FAKE, hs=256, ys=256, os=256,
             xs=256, grow=0, gcol=0, rows=8, hidden=256, ht=0, yt=0, xt=0, gt=0, wt=0, scale=1.0,
             eps=1e-6)
    a.update(over)
    assert lib.moe_reader_residual_norm(BK._NORM.pack(*(a[n] for n in NORM)), None) == RD.EINVAL


def test_residual_norm_of_no_rows(lib):
    args = BK._NORM.pack(*[0] * 13, 0, 64, 0, 0, 0, 0, 0, 1.0, 1e-6)
    assert lib.moe_reader_residual_norm(args, None) == RD.OK
    assert lib.moe_reader_residual_norm(None, None) == RD.EINVAL


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs a C compiler")
def test_packed_structs_match_the_header(tmp_path):
    """Sizes and every field's offset of the argument structs."""
    text = open(os.path.join(ROOT, "include", "moe_reader.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    formats = {"kv_plan": BK._PLAN, "kv_append": BK._APPEND, "kv_attend": BK._ATTEND,
               "kv_select": BK._SELECT, "residual_norm": BK._NORM}
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
            size = struct.calcsize(k)
            lines.append(f'printf("%zu\\n", offsetof(moe_reader_{name}_args, {f}));')
            want.append(at)
            at += size
        lines.append(f'printf("%zu\\n", sizeof(moe_reader_{name}_args));')
        want.append(fmt.size)
    src = tmp_path / "sizes.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"moe_reader.h\"\n"
                   "int main(void) {\n" + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(g) for g in got] == want


def test_operator_cases_are_consistent():
    """The benchmark cases' plain description: names, work and lengths (no GPU)."""
    import importlib.util
    import random

    spec = importlib.util.spec_from_file_location("operator_cases",
                                                  os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    cases = m.listed()
    assert len({c["name"] for c in cases}) == len(cases) <= 12
    rng = random.Random(4)
    for c in cases + [m.draw(rng) for _ in range(50)]:
        w = m.work(c)
        assert w["bytes"] > 0 and w["flops"] > 0
