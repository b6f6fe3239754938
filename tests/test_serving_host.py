"""CPU checks of what stands around the serving calls: the timing reader's ABI and the binding's build."""
import ctypes

import pytest

from qk_norm_rope_gb300 import api

OLD_KINDS = 9  # of st_kernel_times before the serving kernels had kinds of their own


def test_timing_read_fills_nine_kinds_and_no_more():
    """A program compiled against a header without the serving kinds hands in a struct of nine entries each."""
    size = OLD_KINDS * (8 + 8)
    buf = (ctypes.c_ubyte * 512)(*[0xAB] * 512)
    read = api.lib().st_timing_read
    assert read(ctypes.cast(buf, read.argtypes[0])) == api.ST_OK
    assert bytes(buf[:size]) == bytes(size) and bytes(buf[size:]) == b"\xab" * (512 - size)
    assert ctypes.sizeof(api.st_kernel_times) == size


@pytest.mark.parametrize("n", [0, 3, OLD_KINDS, 14, 20])
def test_timing_read_kinds_fills_what_it_is_given(n):
    launches, ms = (ctypes.c_uint64 * 24)(*[7] * 24), (ctypes.c_double * 24)(*[7.0] * 24)
    assert api.lib().st_timing_read_kinds(launches, ms, n) == api.ST_OK
    assert list(launches) == [0] * n + [7] * (24 - n) and list(ms) == [0.0] * n + [7.0] * (24 - n)


def test_timing_read_kinds_refusals():
    launches, ms = (ctypes.c_uint64 * 1)(), (ctypes.c_double * 1)()
    for args in ((None, ms, 1), (launches, None, 1), (launches, ms, -1)):
        assert api.lib().st_timing_read_kinds(*args) == api.ST_ERR_INVALID_ARG
    assert set(api.st_timing_read()) == set(api.KERNEL_KINDS) and len(api.KERNEL_KINDS) == 14


def test_binding_is_kept_apart_by_torch_and_python(monkeypatch, tmp_path):
    """Built with one torch or Python, then with another, then with the first again: each loads its own."""
    import sysconfig
    import types

    import torch

    from qk_norm_rope_gb300 import build
    var = sysconfig.get_config_var
    now = {}

    def compiled(cmd, **_):  # what a compiler would leave: the versions it was run under
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            if "-c" in cmd:
                f.write(f"{now['torch']} {now['abi']}")
            else:
                f.write(open(cmd[cmd.index("-shared") + 1]).read())
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "OUT", str(tmp_path))
    monkeypatch.setattr(build, "BIND", str(tmp_path / "st_bind.so"), raising=False)
    monkeypatch.setattr(build, "build", lambda **_: str(tmp_path / "libst_rope_attn.so"))
    monkeypatch.setattr(build.subprocess, "run", compiled)
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: now["abi"] if n == "SOABI" else var(n))
    for torch_version, abi in (("2.1", "cpython-312-a"), ("2.2", "cpython-312-a"), ("2.1", "cpython-312-a"), ("2.1", "cpython-313-a"),
                               ("2.1", "cpython-312-a")):
        now.update(torch=torch_version, abi=abi)
        monkeypatch.setattr(torch, "__version__", torch_version)
        for _ in range(2):
            assert open(build.build_bind()).read() == f"{torch_version} {abi}"
