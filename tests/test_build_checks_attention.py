"""Checks of the gfx950 code of attention and rotary positions that need no
GPU.

* no packed float32 arithmetic;
* float32 denormals preserved in every kernel (denorm mode 3), IEEE mode on;
* no scratch memory but in the two float32 gradient kernels of heads above 64
  elements, whose results and operands pass the registers;
* loads to LDS: their LDS address is set in M0 right before, nothing else uses
  M0, and no scalar register that a vector instruction wrote is read by one
  before its 5 wait states are over.
"""
import os
import re

import pytest

from point_cloud_tokenization_amd import build as fbuild

SPILLS = ("attention_sink_kernelIfLi128E", "attention_dkv_kernelIfLi128E")


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    at = tmp_path_factory.mktemp("asm")
    names = ("fpstok_attention.hip", "fpstok_rope.hip")
    out = {}
    for n in names:
        path = str(at / (n + ".s"))
        fbuild.device_asm(path, os.path.join(fbuild.CSRC, n))
        out[n] = open(path).read()
    return out


def test_no_packed_fp32(asm):
    for text in asm.values():
        assert re.findall(r"\bv_pk_(?:fma|mul|add)_f32\w*", text) == []


def test_denormals_and_ieee(asm):
    for text in asm.values():
        kernels = re.findall(r"\.amdhsa_kernel\s+(\S+)", text)
        assert len(kernels) >= 6
        assert text.count(".amdhsa_float_denorm_mode_32 3") == len(kernels)
        assert text.count(".amdhsa_ieee_mode 1") == len(kernels)


def test_scratch(asm):
    for text in asm.values():
        for block in re.split(r"\n  - \.", text[text.index("amdhsa.kernels:"):])[1:]:
            name = re.search(r"\.name:\s+(\S+)", block)
            size = re.search(r"\.private_segment_fixed_size:\s+(\d+)", block)
            if name is None or size is None or not name.group(1).startswith("_Z"):
                continue
            if not any(s in name.group(1) for s in SPILLS):
                assert int(size.group(1)) == 0, name.group(1)


def _instructions(text):
    """The instructions of a file in order, comments and directives left out."""
    out = []
    for line in text.splitlines():
        line = line.split(";")[0].strip()
        if line and not line.startswith((".", "//")) and not line.endswith(":"):
            out.append(line)
    return out


def test_loads_to_lds(asm):
    code = _instructions(asm["fpstok_attention.hip"])
    loads = [i for i, x in enumerate(code) if re.match(r"global_load_lds_|buffer_load.*\blds\b", x)]
    assert len(loads) > 100
    set_m0 = set()
    for i in loads:
        assert re.match(r"s_mov_b32 m0, (s\d+|vcc_lo|vcc_hi)$", code[i - 2]), code[i - 2:i + 1]
        set_m0.add(i - 2)
        wait = re.match(r"s_nop (\d+)$", code[i - 1])
        # s_mov counts one wait state, s_nop n counts n + 1
        assert wait and 1 + int(wait.group(1)) + 1 >= 5, code[i - 2:i + 1]
    for i, x in enumerate(code):
        if re.search(r"\bm0\b", x):
            assert i in set_m0, x
