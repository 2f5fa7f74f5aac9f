"""The tests of the products in tiles run in tiles: the launch plan's choice at their sizes, on the host. And bounds of the launch plans."""
import os
import subprocess

import pytest

from mhc_hyper_connection_amd import _binding as B

from experts_tiles import DOWN, FAR, FAR_RESULTS, GLU, LARGE, PRODUCTS, SMALL

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PRODUCT_OP, GLU_OP, DOWN_OP = 0, 1, 2


def test_sizes_run_in_the_tiles_they_are_for(tmp_path):
    exe = tmp_path / "experts_shape"
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "mhc_hyper_connection_amd", "csrc"),
                    os.path.join(ROOT, "tests", "experts_shape.cpp"), "-o", str(exe)], check=True)
    lines, want = [], []
    for x16 in (0, 1):
        for T, K, N, shape in PRODUCTS:
            lines.append((PRODUCT_OP, T, 1, 1, K, N, x16))
            want.append(shape)
        for op, cases in ((GLU_OP, GLU + FAR), (DOWN_OP, DOWN + FAR + FAR_RESULTS)):
            for *size, shape in cases:
                lines.append((op, *size, x16))
                want.append(shape)
    r = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, l)) for l in lines), capture_output=True, text=True, check=True, timeout=60)
    got = [tuple(map(int, l.split())) for l in r.stdout.splitlines()]
    assert len(got) == len(lines)
    for l, w, (valid, shape, units, places) in zip(lines, want, got):
        assert valid == 1 and shape == w, (l, w, shape)
    # each op in both shapes, and workgroups with several units among them
    for op in (PRODUCT_OP, GLU_OP, DOWN_OP):
        assert {w for l, w in zip(lines, want) if l[0] == op} == {SMALL, LARGE}
    assert any(places and units > 2 * places for _, _, units, places in got)


def test_units_of_offsets_of_any_content(tmp_path):
    exe = tmp_path / "experts_units_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I", os.path.join(ROOT, "mhc_hyper_connection_amd", "csrc"), os.path.join(ROOT, "tests", "experts_units_check.cpp"),
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr


def test_the_routings_grid_is_bounded():
    # workgroups of 16 tokens up to 256 experts, of 4 above: 2^26 tokens are 2^24 workgroups of 256 threads there, one more than a grid holds.
    # Within the bound the refusal is that of the missing tensors.
    for E, most in ((256, 1 << 26), (257, (1 << 26) - 4), (1024, (1 << 26) - 4)):
        for call, n in ((B.raw_route, 4), (B.raw_route_backward, 5)):
            for T, status in ((most, B.MHC_ERR_NULLPTR), (most + 1, B.MHC_ERR_PARAM_INVALID)):
                assert call(B.RouteParams(T, E, 2, 1, 1, 2, 0, 1, 2, 1.0), *(None,) * n, None) == status, (E, T)


def test_terms_in_16_bits_are_the_callers_choice():
    size = lambda name, dtype: B.products_workspace_size(name, B.ExpertsParams(8192, 64, 8, 4096, 2048, 0, dtype), True)
    down, glu, pairs, bf16, f16 = "mhc_experts_down", "mhc_experts_glu", 8192 * 8, 0, 1
    assert size(down, bf16) == size(down, f16) == size(down, f16 | B.SHORT_TERMS) == pairs * 4096 * 4       # fp16's are not shortened
    assert size(down, bf16 | B.SHORT_TERMS) == pairs * (4096 * 2 + 4096 // 32)
    assert size(glu, bf16) == size(glu, f16) == 0
    for name, dtype in ((down, 2 | B.SHORT_TERMS), (down, B.SHORT_TERMS << 1), (down, -1), (glu, bf16 | B.SHORT_TERMS), (glu, f16 | B.SHORT_TERMS)):
        with pytest.raises(B.MhcError) as e:
            size(name, dtype)
        assert e.value.status == B.MHC_ERR_PARAM_INVALID, (name, dtype)
