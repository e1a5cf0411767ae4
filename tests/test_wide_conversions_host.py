"""CPU check of the attention's machine code: conversions between 32 values and six-bit codes write
their first results before they have read their last operands, so that the compiler has to know
("early-clobber") that none of their operands may share a register with the result."""
import importlib.util
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    """(the compiler's instructions before registers are given out, the assembly) of attention_kv4.hip"""
    spec = importlib.util.spec_from_file_location("gdn_build", os.path.join(ROOT, "gated_deltanet_token_amd", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    out = tmp_path_factory.mktemp("conversions") / "attention.s"
    r = subprocess.run([build.HIPCC] + build.CFLAGS + ["--cuda-device-only", "-S", "-mllvm", "-print-after=finalize-isel",
                                                       os.path.join(build.CSRC, "attention_kv4.hip"), "-o", str(out)],
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-3000:]
    return r.stdout.splitlines(), out.read_text().splitlines()


def test_the_compiler_keeps_operands_apart_from_results(code):
    """Early clobbers of the compiler's own instructions, and of those that the source writes out."""
    own = [x for x in code[0] if re.search(r"= .*V_CVT_SCALEF32_(PK32|2XPK16)", x)]
    written = [x for x in code[0] if re.search(r"INLINEASM.*v_cvt_scalef32_(pk32|2xpk16)", x)]
    assert own and written
    for x in own:
        assert x.lstrip().startswith("early-clobber"), x
    for x in written:
        assert "regdef-ec:" in x and "regdef:" not in x, x


def registers(operand):
    m = re.fullmatch(r"v\[(\d+):(\d+)\]|v(\d+)", operand)
    return set() if m is None else {int(m[3])} if m[3] else set(range(int(m[1]), int(m[2]) + 1))


def test_no_operand_shares_a_register_with_the_result(code):
    found = 0
    for x in code[1]:
        m = re.match(r"\s*v_cvt_scalef32_(?:pk32|2xpk16)\w*\s+([^;]*)", x)
        if m:
            found += 1
            result, *operands = (registers(y.strip()) for y in m[1].split(", "))
            assert len(result) in (6, 32) and not any(result & y for y in operands), x
    assert found
