"""The 8-bit cache's C ABI from C: include/cfz_kv8.h compiles on its own as C11 and as C++17 with
warnings as errors, and a plain C client links against libcfz.so and meets its refusals and its
workspace sizes without a GPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INC = os.path.join(ROOT, "include")
LIBDIR = os.path.join(ROOT, "diffusion_activation_residual_amd")

CLIENT = r"""
#include "cfz_kv8.h"
#include <stdio.h>
#include <string.h>

static int bad(const char *what) { printf("%s: %s\n", what, cfz_last_error()); return 1; }

int main(void)
{
    /* addresses that nothing reads: every call below is refused or has nothing to do */
    static float scales[8];
    static int32_t ints[8];
    static _Alignas(16) unsigned char memory[16];
    cfz_kv8_cache c = {4, 2, 64, 32, CFZ_KV8_INT8, memory, memory, 0, 0, 0};
    cfz_kv8_batch b = {1, 4, ints, ints, ints, 16, 16};
    cfz_kv8_blocks l = {ints, 2, 8};
    cfz_kv8_rotation r = {scales, scales, 0, 4, 12, 0};
    if (cfz_kv8_append(&c, &b, CFZ_KV8_BF16, memory, memory, 128, 128, 0, 0) != CFZ_ERR_NULL)
        return bad("append without scales");
    if (cfz_kv8_append(&c, &b, CFZ_KV8_BF16, memory, memory, 128, 128, &r, 0) != CFZ_ERR_SHAPE)
        return bad("append with 12 dimensions rotated");
    if (cfz_kv8_gather(&c, &b, (cfz_kv8_dtype)7, memory, memory, 0) != CFZ_ERR_UNSUPPORTED)
        return bad("gather to no type");
    if (cfz_kv8_attend(&c, &b, CFZ_KV8_F16, memory, 128, 2, 0, -1.0f, 128, &l, memory, 128, scales, 0,
                       0, 0) != CFZ_ERR_SHAPE)
        return bad("attend with a negative scale");
    if (cfz_kv8_select(&c, &b, CFZ_KV8_F16, memory, 128, 2, 0, 128, 2, 1, &l, 0, 0, 0) != CFZ_ERR_SHAPE)
        return bad("select of more than count");
    if (!strstr(cfz_last_error(), "count"))
        return bad("the text of the last refusal");
    if (cfz_kv8_select_workspace_bytes(&c, &b, 128, &l) != 2 * 2 * 4 * 8)
        return bad("select workspace");
    if (cfz_kv8_attend_workspace_bytes(&c, &b, 2, 128, 0) != 0)
        return bad("attend workspace");
    b.tokens = 0;
    if (cfz_kv8_append(&c, &b, CFZ_KV8_F32, 0, 0, 128, 128, 0, 0) != CFZ_OK)
        return bad("append of nothing");
    printf("OK\n");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("gcc") is None or shutil.which("g++") is None,
                    reason="gcc/g++ not available")
def test_header_is_self_contained_c_and_cxx(tmp_path):
    for comp, std, ext in (("gcc", "-std=c11", "c"), ("g++", "-std=c++17", "cpp")):
        src = tmp_path / f"inc.{ext}"
        src.write_text('#include "cfz_kv8.h"\nint main(void) { return 0; }\n')
        r = subprocess.run([comp, std, "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", INC,
                            "-c", str(src), "-o", str(tmp_path / f"inc_{ext}.o")],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_c_client_links_and_validates(tmp_path):
    if not os.path.exists(os.path.join(LIBDIR, "libcfz.so")):
        pytest.skip("libcfz.so is not built")
    src, exe = tmp_path / "client.c", tmp_path / "client"
    src.write_text(CLIENT)
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-I", INC, str(src), "-L",
                        LIBDIR, "-lcfz", "-Wl,-rpath," + LIBDIR, "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.strip() == "OK", run.stdout + run.stderr
