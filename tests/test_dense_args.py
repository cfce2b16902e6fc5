"""Where the gated block's calls send their kernels in the kept buffer, up to the most rows that they take: the library's own
objects with the launches replaced, so that sizes of hundreds of GB are checked on the CPU."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
WRAPPED = ["cudaGetDevice", "cudaGetSymbolAddress", "_ZN2la12launch_denseERKNS_9DenseArgsEP11CUstream_st",
           "_ZN2la17launch_gated_gradERKNS_13GatedGradArgsEP11CUstream_st",
           "_ZN2la17launch_dense_pairERKNS_9DenseArgsES2_P11CUstream_st"]


@pytest.fixture(scope="module")
def places(built_lib, tmp_path_factory):
    from linear_attention_chunked_conv1d_gb300 import build
    out = str(tmp_path_factory.mktemp("dense_args") / "places")
    objects = [os.path.join(build.BUILD_DIR, os.path.basename(s)[:-3] + ".o") for s in build.sources()]
    if not all(os.path.exists(o) for o in objects):  # of a library that was built elsewhere
        build.build(force=True)
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, "-o", out,
                    os.path.join(HERE, "dense_args", "places.cu"), *objects, "-lcudart_static",
                    *[a for w in WRAPPED for a in ("-Xlinker", f"--wrap={w}")]], check=True)
    return out


@pytest.mark.parametrize("m,f", [(1, 1), (3, 8), (1000, 333), (1 << 20, 4096), ((1 << 29) - 1, 8), (1 << 29, 24), (1 << 30, 8),
                                 ((1 << 30) + 1, 1), (2 ** 31 - 1024, 8), (2 ** 31 - 1024, 131000), (8, 2 ** 31 - 1024), (1 << 20, 1 << 28)])
def test_the_lower_plane_lies_behind_the_upper_one(places, m, f):
    """gate | up [M][2 whole8(F)]: 16 bits of each in the upper plane, then eight in the lower one."""
    r = subprocess.run([places, str(m), str(f)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    kept, written, read = map(int, r.stdout.split())
    values = m * 2 * ((f + 7) // 8 * 8)
    assert kept == 3 * values and written == read == 2 * values
