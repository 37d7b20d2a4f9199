"""Structural guard on the built gfx950 code of the operators between the
GEMMs, beside tests/test_isa_guard.py: no packed binary32 instruction, no
approximate transcendental or reciprocal outside the expansion of the
correctly rounded division, and no fused multiply-add in the kernels whose
bytes are defined step by step (layer norm's elements, the codes)."""
import os
import re

import pytest

from int8_gemm_amd import build as B
from test_isa_guard import FORBIDDEN, compile_asm, have_hipcc, scan

SOURCES = ["norm.hip", "checkpoint.hip", "logprob.hip"]
KERNELS = ["ln_fwd_kernel", "ln_fwd_long_kernel", "ln_bwd_kernel", "ln_bwd_long_kernel", "ln_bwd_cols_kernel",
           "checkpoint_store_kernel", "checkpoint_read_kernel", "lp_part_kernel", "lp_join_kernel", "lp_bwd_kernel"]
# the exponential is written with fused steps on purpose (GELU's gradient, the
# log probabilities)
FUSED = re.compile(r"checkpoint_read_kernel\w*Li2E|lp_\w+_kernel")

pytestmark = pytest.mark.skipif(not have_hipcc(), reason="hipcc (ROCm) is needed to build the code")


@pytest.fixture(scope="module")
def functions(tmp_path_factory):
    d = tmp_path_factory.mktemp("rowops_asm")
    procs = [(s, str(d / (s + ".s"))) for s in SOURCES]
    procs = [(s, out, compile_asm(os.path.join(B.CSRC, s), out)) for s, out in procs]
    found = {}
    for s, out, p in procs:
        _, err = p.communicate()
        assert p.returncode == 0, f"hipcc -S {s} failed:\n{err[-2000:]}"
        found.update(scan(out))
    return found


@pytest.mark.timeout(600)
def test_every_kernel_is_there(functions):
    names = " ".join(functions)
    assert not [k for k in KERNELS if k not in names]


@pytest.mark.timeout(600)
def test_float_instructions(functions):
    bad = []
    for fn, c in functions.items():
        # binary64 estimates are refined to binary64 precision; binary32 ones are not allowed
        fused = FUSED.search(fn) is not None
        bad += [(fn, op, n) for op, n in c.items()
                if FORBIDDEN.match(op) and not op.endswith("_f64") and not (fused and op == "v_fmaak_f32")]
        n_div = c["v_div_fixup_f32"]
        if c["v_div_fmas_f32"] != n_div or c["v_div_scale_f32"] != 2 * n_div:
            bad.append((fn, "division", dict(c)))
        if not fused:
            for op, n in (("v_fma_f32", 3 * n_div), ("v_fmac_f32", 2 * n_div)):
                if c[op] != n:
                    bad.append((fn, op, c[op], n))
    assert not bad, bad[:10]


@pytest.mark.timeout(600)
def test_in_place_kernels_promise_no_apartness(tmp_path):
    """The kernels for an output that is the input, which take both as
    arguments, must not declare them apart (__restrict__, the compiler's
    noalias): a load could then move behind another value's store."""
    out = str(tmp_path / "checkpoint.ll")
    p = compile_asm(os.path.join(B.CSRC, "checkpoint.hip"), out, ("-emit-llvm",))
    _, err = p.communicate()
    assert p.returncode == 0, err[-2000:]
    with open(out) as f:
        heads = [line for line in f if line.startswith("define ") and "checkpoint_read_kernel" in line]
    apart = [h for h in heads if re.search(r"checkpoint_read_kernel\w*Li[012]ELb1E", h)]
    in_place = [h for h in heads if h not in apart]
    assert len(in_place) == 6 and len(apart) == 9         # 3 types; 2 uses in place, and the restoring one
    assert not [h[:200] for h in in_place if "noalias" in h.split("(", 1)[1]]


@pytest.mark.timeout(600)
def test_every_declared_kernel_is_built(functions):
    """No kernel of the sources is left out of the scanned code, and so none
    stays in them that no call reaches (templates are built where they are used)."""
    names, declared, found = " ".join(functions), set(), 0
    for s in SOURCES:
        with open(os.path.join(B.CSRC, s)) as f:
            text = f.read()
        found += text.count("__global__")
        declared |= set(re.findall(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\s*\(", text))
    assert len(declared) == found and set(KERNELS) <= declared, sorted(declared)
    assert not [k for k in declared if not re.search(rf"\d+{k}(I|E|P|N)", names)]
