"""The compiled argument checks are needed by the speculative step's calls alone:
without them everything else loads and runs, and those calls say what to do."""

import subprocess
import sys

import pytest

WITHOUT = """
import sys

class Block:
    def find_spec(self, name, path=None, target=None):
        if name == "paged_kv_cache_52_gb300._marshal":
            raise ImportError("built for another PyTorch")

sys.meta_path.insert(0, Block())
import torch
from paged_kv_cache_52_gb300 import pagedkv as pk
bm = pk.BlockManager(4, 16)
bm.add_sequence(1, range(20))
assert bm.reserve_draft(1, 3)[0] == [20, 21, 22] and bm.num_free_blocks() == 2
bm.close()
assert pk.status_string(0) == "PKV_OK"
x = torch.zeros(2, dtype=torch.int32)
for call in (lambda: pk.draft_tree_layout(x, x, x, 1),
             lambda: pk.kv_accept_rows(x, x, x, x, x, x, x),
             lambda: pk.qk_norm_rope_append(x, x, x, x, x, x, x, x),
             lambda: pk.paged_tree_attention(x, x, x, x, x, x, x, 1.0, max_q_len=1, workspace=x)):
    try:
        call()
    except RuntimeError as e:
        assert "_marshal.so is not built" in str(e) and "build" in str(e), e
    else:
        raise AssertionError("not refused")
print("done")
"""


@pytest.fixture(scope="module")
def built():
    import os
    from paged_kv_cache_52_gb300 import build as b
    if not (os.path.exists(b.LIB_PATH) and os.path.exists(b.MARSHAL_PATH)):
        b.build()
    return b


def _run(code):
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root,
                          timeout=300)


def test_other_calls_do_not_need_the_compiled_checks(built):
    proc = _run(WITHOUT)
    assert proc.returncode == 0 and proc.stdout.strip() == "done", proc.stderr


def test_the_compiled_checks_refuse_host_tensors(built):
    proc = _run("""
import torch
from paged_kv_cache_52_gb300 import pagedkv as pk
x = torch.zeros(2, dtype=torch.int32)
for _ in range(2):
    for call in (lambda: pk.draft_tree_layout(x, x, x, 1),
                 lambda: pk.kv_accept_rows(x, x, x, x, x, x, x)):
        try:
            call()
        except ValueError:
            continue
        raise AssertionError("not refused")
print("done")
""")
    assert proc.returncode == 0 and proc.stdout.strip() == "done", proc.stderr


def test_a_module_that_does_not_build_leaves_the_library_in_place(built, monkeypatch, tmp_path):
    b = built
    made = []

    def compiles(nvcc, src):
        return src + ".o", ""

    def fails(nvcc):
        raise RuntimeError("no torch headers")

    def link(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").write("library")
        made.append(out)
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b, "LIB_PATH", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(b, "_nvcc", lambda: "nvcc")
    monkeypatch.setattr(b, "_compile", compiles)
    monkeypatch.setattr(b, "_compile_marshal", fails)
    monkeypatch.setattr(b.subprocess, "run", link)
    with pytest.raises(RuntimeError, match=r"(?s)libpagedkv.so is built.*no torch headers"):
        b.build()
    assert len(made) == 1 and (tmp_path / "lib.so").read_text() == "library"
