"""Structural guard on the built gfx950 code of head.hip and embedding.hip,
beside tests/test_rowops_isa.py: no packed binary32 instruction and no
mixed-precision or legacy one; the hardware's exponential in the head's
kernels only, divisions correctly rounded; no fused multiply-add where an
element's value is defined step by step (the embedding's)."""
import os
import re

import pytest

from int8_gemm_amd import build as B
from test_isa_guard import FORBIDDEN, compile_asm, have_hipcc, scan

SOURCES = ["head.hip", "embedding.hip"]
KERNELS = ["head_fwd_kernel", "head_join_kernel", "head_bounds_kernel", "head_prepare_kernel", "head_weights_kernel", "head_grads_kernel",
           "head_finish_kernel", "head_zero_kernel", "embedding_kernel", "embedding_sort_kernel", "embedding_merge_kernel",
           "embedding_sum_kernel", "embedding_join_kernel", "embedding_few_kernel", "embedding_rank_kernel"]

pytestmark = pytest.mark.skipif(not have_hipcc(), reason="hipcc (ROCm) is needed to build the code")


@pytest.fixture(scope="module")
def functions(tmp_path_factory):
    d = tmp_path_factory.mktemp("ends_asm")
    procs = [(s, str(d / (s + ".s"))) for s in SOURCES]
    procs = [(s, out, compile_asm(os.path.join(B.CSRC, s), out)) for s, out in procs]
    found = {}
    for s, out, p in procs:
        _, err = p.communicate()
        assert p.returncode == 0, f"hipcc -S {s} failed:\n{err[-2000:]}"
        found.update(scan(out))
    return found


@pytest.mark.timeout(600)
def test_every_declared_kernel_is_built(functions):
    names, declared, found = " ".join(functions), set(), 0
    for s in SOURCES:
        with open(os.path.join(B.CSRC, s)) as f:
            text = f.read()
        found += text.count("__global__")
        declared |= set(re.findall(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\s*\(", text))
    assert len(declared) == found and declared == set(KERNELS), sorted(declared)
    assert not [k for k in declared if not re.search(rf"\d+{k}(I|E|P|N)", names)]


@pytest.mark.timeout(600)
def test_float_instructions(functions):
    bad = []
    for fn, c in functions.items():
        head = "head_" in fn
        for op, n in c.items():
            if not FORBIDDEN.match(op) or op.endswith("_f64"):
                continue
            if head and op in ("v_exp_f32", "v_fmaak_f32"):
                continue
            bad.append((fn, op, n))
        n_div = c["v_div_fixup_f32"]
        if c["v_div_fmas_f32"] != n_div or c["v_div_scale_f32"] != 2 * n_div:
            bad.append((fn, "division", dict(c)))
        # (the other kernels of embedding.hip hold 64-bit integer divisions, which go through binary32)
        if "embedding_kernel" in fn and (c["v_fma_f32"] or c["v_fmac_f32"] or n_div):
            bad.append((fn, "fused", c["v_fma_f32"], c["v_fmac_f32"]))
    assert not bad, bad[:10]


@pytest.mark.timeout(600)
def test_no_register_is_spilled_in_the_products(functions, tmp_path):
    """A reload from scratch would wait for every load in flight."""
    out = str(tmp_path / "head.s")
    p = compile_asm(os.path.join(B.CSRC, "head.hip"), out)
    _, err = p.communicate()
    assert p.returncode == 0, err[-2000:]
    with open(out) as f:
        spills = re.findall(r"\.name:\s+(\S*head_\w+kernel\S*).*?\.vgpr_spill_count:\s+(\d+)", f.read(), flags=re.S)
    assert len(spills) >= 8 and not [s for s in spills if s[1] != "0"], spills
