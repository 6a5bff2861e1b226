"""The expert-layer entries exist as Python functions (until the library is
loaded) and as the extension module's, which stand in for them: a call that one
accepts, the other has to accept.  And every list of an entry's arguments (the C
header, the ctypes table, the Python function, the extension module) has to say
the same.  No GPU: every call is refused by the library's checks."""
import ctypes
import importlib.machinery
import inspect
import os
import re
import subprocess
import sys

import pytest

import block_scaled_mxfp4_gb300 as mx
from block_scaled_mxfp4_gb300 import build as mxbuild

ENTRIES = ["mxfp4_moe_route", "mxfp4_group_quantize", "mxfp8_group_quantize", "mxfp4_grouped_gemm", "mxfp8_grouped_gemm",
           "mxfp4_grouped_swiglu", "mxfp8_grouped_swiglu", "mxfp4_moe_combine", "mxfp4_moe_ffn"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    mxbuild.build()
    mx.lib()


def forms(name):
    return {"python": mx._python_entries[name], "extension": getattr(mx, name)}


def parameters(name):
    return list(inspect.signature(mx._python_entries[name]).parameters)


@pytest.mark.parametrize("name", ENTRIES)
def test_both_forms_show_the_same(name):
    python, extension = forms(name).values()
    assert type(extension).__name__ == "builtin_function_or_method" and inspect.isfunction(python)
    assert str(inspect.signature(python)) == str(inspect.signature(extension))
    assert python.__doc__ == extension.__doc__


@pytest.mark.parametrize("name", ENTRIES)
def test_header_table_and_python_agree(name):
    text = re.sub(r"/\*.*?\*/", "", open(mx.HEADER).read(), flags=re.S)
    declared = re.search(r"\bint\s+%s\s*\(([^)]*)\)" % name, text).group(1).split(",")
    names = [re.search(r"(\w+)\s*$", d).group(1) for d in declared]
    kinds = {"int64_t": ctypes.c_int64, "size_t": ctypes.c_size_t, "float": ctypes.c_float, "int": ctypes.c_int}
    types = [ctypes.c_void_p if "*" in d else kinds[d.replace("const", "").split()[0]] for d in declared]
    assert names == parameters(name) and types == list(getattr(mx.lib(), name).argtypes)


@pytest.mark.parametrize("form", ["python", "extension"])
@pytest.mark.parametrize("name", ENTRIES)
def test_arguments_by_name(name, form):
    call, names = forms(name)[form], parameters(name)
    # Zeros and null pointers: everything converts, and the library refuses the sizes.
    values = {n: 0 for n in names}
    n = len(names)
    for by_place in (0, 1, n // 2, n - 1, n):
        with pytest.raises(mx.Mxfp4Error) as e:
            call(*list(values.values())[:by_place], **{k: values[k] for k in reversed(names[by_place:])})
        assert name in str(e.value) and e.value.status == -1
    for args, kw in (((), dict(values, more=1)),                                             # an unknown name
                     ((), {k: values[k] for k in names if k not in (names[3], "stream")}),   # one missing
                     ((0,), values),                                                         # one twice
                     ((0,) * (n + 1), {}), ((0,) * n, dict(stream=0)), ((), {})):
        with pytest.raises(TypeError):
            call(*args, **kw)


@pytest.mark.parametrize("name", ENTRIES)
def test_each_argument_reaches_its_place(name):
    """A value of the wrong type is refused under every name, so none is dropped."""
    names = parameters(name)
    for wrong in names:
        with pytest.raises((TypeError, AttributeError)):
            getattr(mx, name)(**{n: object() if n == wrong else 0 for n in names})


WITHOUT = """
import warnings
from block_scaled_mxfp4_gb300 import build
import block_scaled_mxfp4_gb300 as mx
build.BINDING_LIB = {path!r}
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    mx.lib()
assert len(seen) == 1 and "marshalled in Python" in str(seen[0].message), seen
assert mx.mxfp4_version() > 0 and mx.mxfp4_gemm_workspace_size(128, 256, 512) >= 0
for call, args in ((mx.mxfp4_gemm, [0] * 20), (mx.mxfp4_moe_combine, [0] * 19)):
    try:
        call(*args, stream=0)
    except mx.Mxfp4Error as e:
        assert e.status == -1
    else:
        raise AssertionError
print("fine")
"""


@pytest.mark.parametrize("content", [None, b"", b"\x7fELF of another machine"])
def test_the_library_works_without_the_extension(tmp_path, content):
    path = tmp_path / "_entry.so"
    if content is not None:
        path.write_bytes(content)
    run = subprocess.run([sys.executable, "-c", WITHOUT.format(path=str(path))], cwd=os.path.dirname(os.path.dirname(mx.__file__)),
                         capture_output=True, text=True)
    assert run.returncode == 0 and run.stdout == "fine\n", run.stderr


def test_build_goes_on_without_the_extension(tmp_path, monkeypatch):
    monkeypatch.setattr(mxbuild, "BINDING_LIB", str(tmp_path / "_entry.so"))
    monkeypatch.setenv("PATH", str(tmp_path))              # no compiler
    with pytest.warns(UserWarning, match="marshalled in Python"):
        assert mxbuild.build() == mxbuild.LIB
    monkeypatch.undo()
    source = tmp_path / "binding.c"
    source.write_text("#error no headers\n")
    monkeypatch.setattr(mxbuild, "BINDING_LIB", str(tmp_path / "_entry.so"))
    monkeypatch.setattr(mxbuild, "BINDING_SRC", str(source))
    with pytest.warns(UserWarning, match="marshalled in Python"):
        assert mxbuild.build() == mxbuild.LIB


def test_the_extension_is_named_for_its_interpreter():
    assert any(mxbuild.BINDING_LIB.endswith(s) for s in importlib.machinery.EXTENSION_SUFFIXES if s != ".so")
    assert mx.mxfp4_moe_ffn.__module__ == "block_scaled_mxfp4_gb300._entry"
