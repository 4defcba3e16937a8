"""Rotation tables are read as read-only data by the compressor's kernels, so the kernel that builds one lets no kernel behind
it start early."""
import os

ROTARY = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deepseek_v4_sparse_c128_gb300", "csrc", "c128_rotary.cu")


def test_building_a_table_lets_no_kernel_start_early():
    code = open(ROTARY).read()
    start = code.index("cos_sin_kernel(const __grid_constant__")
    body = code[start:code.index("\n}\n", start)]
    assert "grid_dependency_wait()" in body and "launch_dependents" not in body
    assert "launch_dependents" in code[code.index("rotate_kernel(const RotateParams"):]
