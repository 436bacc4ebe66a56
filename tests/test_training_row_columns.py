"""Columns that a thread of the SiLU * up backward visits, for every width that the entry point takes: the loop is taken
out of the kernel's source and compiled for the CPU."""
import os
import re
import subprocess

import pytest

from _util import ROOT

SRC = open(os.path.join(ROOT, "mixture_experts_routed_route_amd", "csrc", "grad_rows.hip")).read()


def loop():
    """The loop's head and its column, as the kernel has them, and the limit that the head names."""
    body = SRC[SRC.index("void silu_mul_backward_kernel("):]
    head = re.search(r"for \(\w+ c0 = [^;]*; c0 < \w+; c0 \+= [^)]*\)", body).group(0)
    column = set(re.findall(r"const \w+ c = c0 \+ [^;]*;", body[:body.index("#pragma unroll\n    for (int o")]))
    assert len(column) == 1
    tests = set(re.findall(r"if \((c (?:<|>=) \w+)\)", body))
    limit = re.search(r"c0 < (\w+);", head).group(1)
    assert tests == {f"c < {limit}", f"c >= {limit}"}
    declared = re.search(rf"const (\w+) {limit} = [^;]*;", body[:body.index(head)])
    return head, column.pop(), declared.group(0) if declared else "", limit


@pytest.mark.parametrize("tpr", [64, 256])
def test_columns_of_a_thread(tpr, tmp_path):
    """Every eighth column of a thread's share once and none outside the row, up to the widest row (2^31 - 8)."""
    head, column, declared, limit = loop()
    (tmp_path / "columns.cpp").write_text(f"""
#include <cstdint>
#include <cstdio>
#include <initializer_list>
static bool visits(int n, int t) {{
    constexpr int TPR = {tpr};
    {declared}
    int64_t seen = 0, last = t * 8 - TPR * 8;
    {head} {{
        for (int b = 0; b < 2; ++b) {{
            {column}
            if (!(c < {limit})) continue;
            const int64_t at = c;
            if (at != last + TPR * 8 || at < 0 || at + 8 > n) return false;
            last = at;
            ++seen;
        }}
        if (seen > (int64_t(1) << 28)) return false;
    }}
    const int64_t want = t * 8 < n ? (int64_t(n) - t * 8 + TPR * 8 - 1) / (TPR * 8) : 0;
    return seen == want;
}}
int main() {{
    const int widths[] = {{8, 16, 504, 512, 1024, 2048, 2056, 4096, 14336, 1 << 20, 1 << 30, INT32_MAX - 8191, INT32_MAX - 4095,
                          INT32_MAX - 4087, INT32_MAX - 2047, INT32_MAX - 15, INT32_MAX - 7}};
    for (int n : widths)
        for (int t : {{0, 1, TPRS / 2, TPRS - 1}})
            if (!visits(n, t)) {{
                std::printf("n %d thread %d\\n", n, t);
                return 1;
            }}
    return 0;
}}
""".replace("TPRS", str(tpr)))
    exe = tmp_path / "columns"
    subprocess.run(["g++", "-O1", "-fwrapv", "-o", exe, tmp_path / "columns.cpp"], check=True, timeout=60)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
