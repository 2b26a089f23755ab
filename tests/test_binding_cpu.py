"""How _binding.so is built and loaded (CPU only)."""
import os
import subprocess
import sys

import pytest

from conftest import ROOT

from top_sparse_attention_qsa_b200 import build as B


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_only_the_calls_that_need_it_load_it():
    """A binding that does not load stops the appends and the 4-bit attention, not the package."""
    r = run("import sys\n"
            "sys.modules['top_sparse_attention_qsa_b200._binding'] = None     # as an undefined symbol would\n"
            "import torch\n"
            "import top_sparse_attention_qsa_b200 as qsa\n"
            "assert qsa.abi_version() >= 1\n"
            "q, i = torch.zeros(2, 3, 256, dtype=torch.bfloat16), torch.zeros(2, 1, 4, dtype=torch.int32)\n"
            "try:\n"
            "    qsa.sparse_prefill_fwd(q, q, q, i)\n"
            "except ValueError:\n"                       # a host tensor, seen by the call itself
            "    pass\n"
            "cache = qsa.fp4_cache(4, 1, device='cpu')\n"
            "for f in (lambda: qsa.kv_append(q, q, i, i, None, q, q), lambda: qsa.sparse_decode_fp4_fwd(q, cache, i, 1., 1.)):\n"
            "    try:\n"
            "        f()\n"
            "    except ImportError as e:\n"
            "        assert 'build it again' in str(e)\n"
            "    else:\n"
            "        raise AssertionError('no error')\n")
    assert r.returncode == 0, r.stderr


def test_a_missing_binding_is_named(tmp_path):
    r = run("from top_sparse_attention_qsa_b200 import _capi\n"
            f"_capi.BINDING_PATH = {os.path.join(str(tmp_path), '_binding.so')!r}\n"
            "try:\n"
            "    _capi._binding.kv_append\n"
            "except ImportError as e:\n"
            "    assert 'is missing: build it with' in str(e)\n"
            "else:\n"
            "    raise AssertionError('no error')\n")
    assert r.returncode == 0, r.stderr


def test_libraries_are_built_before_the_binding(monkeypatch):
    """A binding that cannot be built leaves both libraries in place."""
    made = []
    monkeypatch.setattr(B, "_build_one", lambda lib, *a: made.append(lib))

    def fail(force):
        raise RuntimeError("no headers")

    monkeypatch.setattr(B, "_build_binding", fail)
    with pytest.raises(RuntimeError):
        B.build()
    assert made == [B.LIB, B.DEBUG_LIB]
    assert B.build(binding=False) == B.LIB


def test_a_binding_of_another_torch_is_built_again(monkeypatch, tmp_path):
    """What the binding was compiled against decides beside the file times."""
    B.build()
    assert B.binding_up_to_date()
    with open(B.BINDING_ABI) as f:
        assert f.read() == B.binding_abi()
    note = tmp_path / "abi"
    monkeypatch.setattr(B, "BINDING_ABI", str(note))
    assert not B.binding_up_to_date()                    # no note: built before there was one
    note.write_text(B.binding_abi())
    assert B.binding_up_to_date()
    import torch
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert not B.binding_up_to_date()
