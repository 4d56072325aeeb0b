"""How the library and the binding's module are built (no GPU; the compilers are
stand-ins that write down how they were called)."""
import os
import stat
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def stand_in(path, log):
    """A compiler that makes its -o file and logs its arguments."""
    path.write_text(f"""#!{sys.executable}
import sys
open({str(log)!r}, "a").write(" ".join(sys.argv) + "\\n")
open(sys.argv[sys.argv.index("-o") + 1], "w").close()
""")
    path.chmod(path.stat().st_mode | stat.S_IXUSR)


def run(code, tmp_path, **env):
    head = ("from hadamard_rotated_bit_fwht_b200 import build\n"
            f"build.LIB = {str(tmp_path / 'libkvq.so')!r}\n"
            f"build.BIND = {str(tmp_path / 'kvq_bind.so')!r}\n"
            f"build.OBJ_DIR = {str(tmp_path / 'obj')!r}\n")
    return subprocess.run([sys.executable, "-c", code.replace("HEAD\n", head)], cwd=ROOT,
                          env={**os.environ, **env}, capture_output=True, text=True, timeout=300)


def test_the_library_needs_no_torch(tmp_path):
    stand_in(tmp_path / "nvcc", tmp_path / "log")
    r = run("import sys\nsys.modules['torch'] = None\nHEAD\nprint(build.build(force=True))", tmp_path,
            NVCC=str(tmp_path / "nvcc"))
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == str(tmp_path / "libkvq.so")
    assert (tmp_path / "libkvq.so").exists() and not (tmp_path / "kvq_bind.so").exists()
    assert "binding is not built" in r.stderr
    calls = (tmp_path / "log").read_text().splitlines()
    assert sum(" -c " in c for c in calls) == len(calls) - 1 > 1


def test_nvcc_by_name(tmp_path):
    """A name on the PATH, a link, and a path: the headers beside the compiler."""
    cuda = tmp_path / "cuda"
    for d in ("bin", "include"):
        (cuda / d).mkdir(parents=True)
    stand_in(cuda / "bin" / "nvcc", tmp_path / "log")
    (cuda / "include" / "cuda_runtime_api.h").write_text("")
    (tmp_path / "links").mkdir()
    (tmp_path / "links" / "nvcc").symlink_to(cuda / "bin" / "nvcc")
    stand_in(tmp_path / "links" / "g++", tmp_path / "gxx")
    for nvcc, path in (("nvcc", cuda / "bin"), ("nvcc", tmp_path / "links"),
                       (str(cuda / "bin" / "nvcc"), tmp_path), (str(tmp_path / "links" / "nvcc"), tmp_path)):
        r = run("HEAD\nbuild.build_bind(force=True)", tmp_path, NVCC=nvcc,
                PATH=f"{path}:{tmp_path / 'links'}:{os.environ['PATH']}")
        assert r.returncode == 0, r.stderr
    for call in (tmp_path / "gxx").read_text().splitlines():
        assert f"-I{cuda / 'include'}" in call.split()
    r = run("HEAD\nbuild.build_bind(force=True)", tmp_path, NVCC=str(tmp_path / "none" / "nvcc"))
    assert r.returncode and "cuda_runtime_api.h" in r.stderr


def test_a_module_of_another_torch_is_stale(tmp_path):
    from hadamard_rotated_bit_fwht_b200 import build
    build.build_bind()
    key = build.bind_key()
    assert build.bind_is_for(key)
    assert not build.bind_is_for(key[:-1]) and not build.bind_is_for(key + "x")
    # not loaded, and built again
    code = ("HEAD\nbuild.BIND = {bind!r}\nbuild.bind_key = lambda: 'kvq_bind for another torch'\n"
            "from hadamard_rotated_bit_fwht_b200 import kvq\n"
            "try:\n    kvq.bind()\nexcept ImportError as e:\n    print('refused', e)\n"
            "build.BIND = {copy!r}\nbuild.build_bind()\n")
    copy = tmp_path / "copy.so"
    copy.write_bytes(open(build.BIND, "rb").read())
    os.utime(copy)  # newer than its sources
    stand_in(tmp_path / "g++", tmp_path / "gxx")
    r = run(code.format(bind=build.BIND, copy=str(copy)), tmp_path,
            PATH=f"{tmp_path}:{os.environ['PATH']}")
    assert r.returncode == 0, r.stderr
    assert r.stdout.startswith("refused") and "another Python or torch" in r.stdout
    call, = (tmp_path / "gxx").read_text().splitlines()
    assert '-DKVQ_BIND_KEY="kvq_bind for another torch"' in call
