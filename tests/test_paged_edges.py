"""Paged-cache operators, host side (no GPU): refusals of calls that would pair rows with wrong sequences or write an
output over itself, and the build's bookkeeping."""
import pytest

import persistent_monokernel_decode_gb300 as kie
from test_paged_host import SOME, append_args, attention_args, refused


@pytest.fixture(scope="module", autouse=True)
def built():
    kie.build()
    yield


@pytest.mark.parametrize("change,word", [
    (dict(seqs=SOME, lens=None), "together"), (dict(positions=SOME, lens=None), "together"),
    (dict(seqs=SOME, positions=SOME), "either"), (dict(lens=None), "either"),
    (dict(seqs=SOME, positions=SOME, lens=None, n_table=-1), "n_table"),
    (dict(seqs=SOME, positions=SOME, lens=None, n_table=2, table_stride=3), "table_stride"),
    (dict(seqs=SOME + 2, positions=SOME, lens=None), "aligned"), (dict(seqs=SOME, positions=SOME + 1, lens=None), "aligned")])
def test_attention_of_rows_refuses(change, word):
    a = attention_args()
    for k, v in change.items():
        setattr(a, k, v)
    refused("kie_paged_attention", a, word)


@pytest.mark.parametrize("out_stride", [(512, 64), (256, 128), (64, 256)])
def test_attention_in_place_needs_equal_strides(out_stride):
    """Another block would read a query that this one has overwritten."""
    a = attention_args()
    a.q_stride[:], a.out_stride[:] = (256, 64), out_stride
    refused("kie_paged_attention", a, "strides")


@pytest.mark.parametrize("out_stride", [(0, 64), (256, 0)])
def test_attention_refuses_an_expanded_output(out_stride):
    a = attention_args()
    a.out, a.q_stride[:], a.out_stride[:] = 2 * SOME, (256, 64), out_stride
    refused("kie_paged_attention", a, "stride of 0")


def strided_append_args(dtype=0):
    a = append_args(dtype)
    a.q_out = 2 * SOME
    for s in (a.q_stride, a.q_out_stride):
        s[:] = (256, 64)
    for s in (a.pages.k_scale_stride, a.pages.v_scale_stride):
        s[:] = (32, 16, 1)
    return a


@pytest.mark.parametrize("name", ["k_stride", "v_stride", "k_scale_stride", "v_scale_stride"])
@pytest.mark.parametrize("dim", [0, 1, 2])
def test_append_refuses_expanded_pages(name, dim):
    a = strided_append_args(3)
    getattr(a.pages, name)[dim] = 0
    refused("kie_paged_append", a, "stride of 0")


@pytest.mark.parametrize("dim", [0, 1])
def test_append_refuses_an_expanded_output(dim):
    a = strided_append_args()
    a.q_out_stride[dim] = 0
    refused("kie_paged_append", a, "stride of 0")


# ---- the build -----------------------------------------------------------------------------------------------

@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """build() with stand-ins for the compilers, its outputs in a folder of the test's; returns what has run."""
    ran = []
    lib, binding = tmp_path / "libkie.so", tmp_path / "_paged.so"
    monkeypatch.setattr(kie, "_BUILD", str(tmp_path))
    monkeypatch.setattr(kie, "LIB_PATH", str(lib))
    monkeypatch.setattr(kie, "BINDING_PATH", str(binding))
    monkeypatch.setattr(kie, "BINDING_ENV_PATH", str(tmp_path / "_paged.env"))
    monkeypatch.setattr(kie, "compile_cmds", lambda: ran.append("lib") or [["true"]])
    monkeypatch.setattr(kie, "link_cmd", lambda: ["touch", str(lib)])
    monkeypatch.setattr(kie, "binding_cmd", lambda: ran.append("binding") or ["touch", str(binding)])
    return ran


def test_build_compiles_what_is_missing_or_old(elsewhere):
    import os
    kie.build()
    assert sorted(elsewhere) == ["binding", "lib"]
    kie.build()
    assert len(elsewhere) == 2
    os.remove(kie.BINDING_PATH)
    kie.build()
    assert elsewhere[2:] == ["binding"] and os.path.exists(kie.BINDING_PATH)
    os.utime(kie.LIB_PATH, (0, 0))
    kie.build()
    assert elsewhere[3:] == ["lib"]
    kie.build(force=True)
    assert sorted(elsewhere[4:]) == ["binding", "lib"]


def test_a_binding_of_another_pytorch_is_compiled_anew(elsewhere, monkeypatch):
    import torch
    kie.build()
    monkeypatch.setattr(torch, "__version__", "0.0")
    kie.build()
    assert elsewhere[2:] == ["binding"]
    kie.build()
    assert len(elsewhere) == 3


@pytest.mark.parametrize("cmd", [["false"], ["/nowhere/g++"]])
def test_the_library_is_complete_where_the_binding_does_not_compile(elsewhere, monkeypatch, cmd):
    import os
    monkeypatch.setattr(kie, "binding_cmd", lambda: cmd)
    with pytest.raises(RuntimeError, match="is built"):
        kie.build()
    assert os.path.exists(kie.LIB_PATH)
    with pytest.raises(RuntimeError):  # and it is not taken for built the next time
        kie.build()


def test_without_pytorch_the_library_alone_is_built(elsewhere, monkeypatch):
    import os
    import sys
    monkeypatch.setitem(sys.modules, "torch", None)
    kie.build()
    kie.build()
    assert elsewhere == ["lib"] and os.path.exists(kie.LIB_PATH) and not os.path.exists(kie.BINDING_PATH)
