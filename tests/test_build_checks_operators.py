"""Checks of the gfx950 code of attention with a learned bias and of the
residual step that need no GPU.

* no packed float32 arithmetic, float32 denormals kept, IEEE mode on;
* scratch memory only where the named kernels' results and operands pass the
  registers, and in no more than they hold now;
* no float32 atomics (their order would change results);
* loads to LDS: their LDS address is set in M0 right before, nothing else uses
  M0, and no scalar register that a vector instruction wrote is read by one
  before its 5 wait states are over.
"""
import os
import re

import pytest

from point_cloud_tokenization_amd import build as fbuild

ATTENTION = ("fpstok_attention_bias.hip", "fpstok_attention_plane.hip")
# bytes a thread at most, by the kernel's name
SPILLS = (
    # float32 heads above 64 elements: results and operands pass the registers
    (r"attention_sink_kernelIfLi128E", 904),
    (r"attention_dkv_kernelIfLi128E", 200),
    # three waves a scheduler, which is worth more than the registers
    (r"attention_few_kernel", 116),
    (r"attention_sink_kernelIDF16b?_?Li64E", 116),
    (r"attention_kernelIDF16b?_?Li(64|128)E.*BiasFromE[12]E", 48),
    # a workgroup of over 512 threads: 128 or 168 registers each
    (r"residual_grad_kernel.*ELi8ELi(768|1024)E", 376),
    (r"residual_grad_kernel.*ELi4ELi1024E", 36),
)


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    at = tmp_path_factory.mktemp("asm")
    out = {}
    for n in ATTENTION + ("fpstok_residual.hip",):
        path = str(at / (n + ".s"))
        fbuild.device_asm(path, os.path.join(fbuild.CSRC, n))
        out[n] = open(path).read()
    return out


def test_arithmetic(asm):
    for text in asm.values():
        assert re.findall(r"\bv_pk_(?:fma|mul|add)_f32\w*", text) == []
        assert re.findall(r"\b(?:ds|global|flat)_(?:atomic_)?(?:pk_)?add_(?:rtn_)?f\w+", text) == []
        kernels = re.findall(r"\.amdhsa_kernel\s+(\S+)", text)
        assert len(kernels) >= 20
        assert text.count(".amdhsa_float_denorm_mode_32 3") == len(kernels)
        assert text.count(".amdhsa_ieee_mode 1") == len(kernels)


def test_scratch(asm):
    seen = 0
    for text in asm.values():
        for block in re.split(r"\n  - \.", text[text.index("amdhsa.kernels:"):])[1:]:
            name = re.search(r"\.name:\s+(\S+)", block)
            size = re.search(r"\.private_segment_fixed_size:\s+(\d+)", block)
            if name is None or size is None or not name.group(1).startswith("_Z"):
                continue
            seen += 1
            most = max([n for p, n in SPILLS if re.search(p, name.group(1))], default=0)
            assert int(size.group(1)) <= most, name.group(1)
    assert seen > 100


def _instructions(text):
    """The instructions of a file in order, comments and directives left out."""
    out = []
    for line in text.splitlines():
        line = line.split(";")[0].strip()
        if line and not line.startswith((".", "//")) and not line.endswith(":"):
            out.append(line)
    return out


@pytest.mark.parametrize("name", ATTENTION)
def test_loads_to_lds(asm, name):
    code = _instructions(asm[name])
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
