"""The offsets at which the bf16 and 8-bit products' kernels read, for every lane of every copy of tiles of all sizes
(compiled for the host: a read past a buffer's end shows in no result)."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "combine_moe_layout_02_amd", "csrc")


def test_copies_stay_inside_their_buffers(tmp_path):
    exe = str(tmp_path / "product_copies")
    subprocess.run(["g++", "-std=c++17", "-O2", "-D__device__=", "-D__forceinline__=inline", "-I", CSRC,
                    os.path.join(HERE, "product_copies_main.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout.split()[0]) > 1_000_000
