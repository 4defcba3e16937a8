"""What a call reads of memory that an earlier kernel of the library may still be writing when its own kernels start
(build_slot_maps and extend_block_tables let their successor start early) is not read as read-only data: such a load is
defined only for memory that nobody writes while the kernel is resident."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deepseek_v4_sparse_c128_gb300", "csrc")


def test_only_rotation_tables_are_read_by_ldg():
    """__ldg on the rows of the cos/sin table (constants of the model), nowhere else; and no parameter is marked as
    read-only to the compiler but the read probe's, whose launches are not early ones."""
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        code = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__ldg\(([^;]*?)\)", code):
            assert re.match(r"(m\.)?cs(_row)?( |$)", m.group(1)), (os.path.basename(path), m.group(0))
            seen += 1
        if not path.endswith("c128_probe.cu"):
            assert "__restrict__" not in code and "ld.global.nc" not in code, path
    assert seen > 0
