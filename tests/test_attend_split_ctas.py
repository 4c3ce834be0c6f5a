"""The split of test_attend_split.py over as many CTAs as the kernel takes: its own lines that bound their number (fewer than
there are when the segments are few) are compiled in place of the test's."""

import os
import re
import shutil
import subprocess

import pytest

import test_attend_split as split


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_work_split_over_the_kernels_own_number_of_ctas(tmp_path):
    with open(os.path.join(split.CSRC, "pa_attend.cuh")) as f:
        common = f.read()
    with open(os.path.join(split.CSRC, "pa_attend_tc.cuh")) as f:
        tc = f.read()
    lines = split._between(tc, "const int want =", "WarpFrag* const wf")
    assert "balanced" in lines and "const int nw =" in lines
    main = split.MAIN
    old = re.search(r"const int want = [^;]*;", main).group(0)
    assert old.count("nw = ") == 1
    main = main.replace(old, """
    const int groups = grid;
    p.max_segments = static_cast<float>(S) * a.num_kv_heads * ((a.max_q_len * a.group + rpt - 1) / rpt);
""" + lines)
    code = split.PRELUDE.replace("FRAG_COST", re.search(r"kFragCost = (\d+);", tc).group(1))
    code = code.replace("int paired, seg_rows; };", "int paired, seg_rows; float max_segments; };").replace("#include <cstdint>", "#include <cmath>\n#include <cstdint>")
    code += split._between(common, "struct SeqView", "// softcap * tanh")
    code += split._between(tc, "__host__ __device__ __forceinline__ int stream_rows", "// A warp's iterator").replace("struct WarpFrag", "struct Unused")
    code += split._between(tc, "__device__ __forceinline__ bool advance_frag", "// The warp's next fragment")
    code += split._between(tc, "// CTA whose range holds", "template <")
    code += main
    src = tmp_path / "split.cpp"
    src.write_text(code)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", str(src), "-o",
                    str(tmp_path / "split")], check=True)
    r = subprocess.run([str(tmp_path / "split")], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
