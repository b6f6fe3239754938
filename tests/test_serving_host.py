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


@pytest.mark.parametrize("mistake", ["chain", "no self", "zero"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_attention_bound_finds_planted_mistakes(dtype, mistake):
    """The bound that cached attention is held to is far below what a wrong mask or a missing result changes."""
    import torch

    import _serving as R
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[dtype]
    B, T, H, Hkv, page, lens = 3, 10, 4, 2, 16, [0, 37, 250]
    full = [n + T for n in lens]
    k, v, pages = R.make_cache(B, full, Hkv, page, dt, 1, fill=0.0)
    R.fill_prefix(k, v, pages, full, 2)
    q = torch.randn(B, T, H, 128, generator=torch.Generator().manual_seed(3)).to(dt)
    parents = R.tree(B, T, 3, 4)
    o, _, bound, _ = R.attention(q, k, v, pages, lens, None, parents)
    if mistake == "chain":
        wrong = R.attention(q, k, v, pages, lens, None, None)[0]
    elif mistake == "zero":
        wrong = torch.zeros_like(o)
    else:  # the last node's own key taken from another row
        k2 = k.clone()
        for b in range(B):
            pg, row = R.slots(pages, page, b, torch.tensor([lens[b] + T - 1, lens[b]]))
            k2[pg[0], row[0]] = k[pg[1], row[1]]
        wrong = R.attention(q, k2, v, pages, lens, None, parents)[0]
    changed = (wrong - o).abs() > 0
    assert changed.any()
    # The last node's own key is one of up to 260 of its row, so that its weight moves outputs by 0.4%, the size of the
    # bf16 bound: some elements have to be found. The others change whole rows: most have to be.
    share = 0.0 if mistake == "no self" else 0.5
    for b in range(B):
        found = ((wrong[b] - o[b]).abs() > bound[b])[changed[b]]
        assert found.double().mean() > share, (b, float(found.double().mean()))


@pytest.mark.parametrize("dim", [0, 1, 2])
def test_outputs_must_not_be_expanded(dim):
    """An output whose rows lie in one place (q itself, broadcast over heads, as q_rot) would keep any of them."""
    from test_abi import FAKE, T
    from test_serving_abi import check
    strides = [5 * 8 * 128, 8 * 128, 128, 1]
    strides[dim] = 0
    check("append", api.ST_ERR_ALIGN, "q_rot must not be expanded", q_rot=T([2, 5, 8, 128], strides=strides))
    check("attn", api.ST_ERR_ALIGN, "o must not be expanded", o=T([2, 5, 8, 128], data=FAKE + (1 << 30), strides=strides))
    one = dict(B=1, T_=1, H=1, Hkv=1)  # a stride of nothing is no expansion
    import torch
    if not torch.cuda.is_available():
        check("append", api.ST_ERR_CUDA, sizes=one, q_rot=T([1, 1, 1, 128], strides=[0, 0, 0, 1]))
