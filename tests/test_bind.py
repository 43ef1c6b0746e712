"""The C++ marshalling of the paged cache's wrappers: its build, and what happens without it (no GPU needed)."""
import importlib.metadata
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_WITHOUT = """
import sys
class Block:
    def find_spec(self, name, path=None, target=None):
        if name == "sliding_window_attention_tcgen05_b200._bind":
            raise ImportError("undefined symbol: some_function_of_another_torch")
sys.meta_path.insert(0, Block())
import torch
import sliding_window_attention_tcgen05_b200 as vx
vx.Workspace(256, device="cpu")
assert vx.lib.vx_swa_attn_workspace(1, 8, 6000, 32, 64, 0) == 1024
cache = vx.PagedCache(1, 4, 16, 2, 64, 1, 4, device="cpu")
x, i = torch.zeros(1, 2, 64), torch.zeros(2, dtype=torch.int32)
for call in (lambda: vx.rope_fwd(x, i.long()), lambda: vx.paged_append(cache, 0, x, x, i, 1),
             lambda: vx.paged_attn_fwd(cache, 0, x, i, 1), lambda: vx.paged_advance(cache, i, 1, 1),
             lambda: vx.paged_evict(cache, 1, 1)):
    try:
        call()
    except ImportError as e:
        assert "some_function" in str(e) and "build.py" in str(e), e
    else:
        raise AssertionError("no error")
print("fine")
"""


def test_the_encoders_calls_do_not_need_it():
    p = subprocess.run([sys.executable, "-c", _WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.strip() == "fine", p.stderr[-2000:]


def test_it_is_rebuilt_for_another_torch(tmp_path, monkeypatch):
    from sliding_window_attention_tcgen05_b200 import build
    runs = []

    class Ok:
        returncode, stdout, stderr = 0, "", ""

    def compiler(cmd, **kw):
        runs.append(cmd)
        open(build.BIND, "w").close()
        return Ok

    monkeypatch.setattr(build, "BIND", str(tmp_path / "_bind.so"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build.subprocess, "run", compiler)
    build.build_bind()
    build.build_bind()
    assert len(runs) == 1
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "99.0")
    build.build_bind()
    build.build_bind()
    assert len(runs) == 2
    Ok.returncode = 1                              # a failed build is tried again
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "99.1")
    for n in (3, 4):
        try:
            build.build_bind()
        except RuntimeError:
            pass
        assert len(runs) == n


def test_a_cache_in_use_is_copied_and_pickled():
    import copy
    import pickle

    import torch

    import sliding_window_attention_tcgen05_b200 as vx
    a = vx.PagedCache(1, 4, 16, 2, 64, 1, 4, weights=True, device="cpu")
    a.table[0, 0] = 3
    object.__setattr__(a, "_described", lambda: None)    # what a call leaves there cannot be pickled
    for b in (copy.deepcopy(a), pickle.loads(pickle.dumps(a))):
        assert b._described is None and a._described is not None
        assert torch.equal(a.table, b.table) and a.table.data_ptr() != b.table.data_ptr()
    b = copy.copy(a)
    assert b._described is None and b.table is a.table
