"""The binding's two libraries: the codec needs libkvq.so alone, and a torch
side that is missing, or made for another torch, is an ImportError of the
paged calls (no GPU needed)."""
import os
import shutil
import subprocess
import sys

import pytest

PKG = "kv_cache_quantization_02_b200"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = f"""
from {PKG} import kvq
assert kvq.kvq_version() >> 16 == 1
assert kvq.kvq_quantize(0, 0, 0, 4, 100, 32, 0, 0) == kvq.KVQ_ERR_DIM
assert kvq.kvq_paged_write(0, 0, 0, 0, 0, 0, 0, 0, 1, 1, 1, 1, 100, 16, 0, 1, 0, 0, 0, 0) == kvq.KVQ_ERR_DIM
for call in (lambda: kvq.paged_write(*[None] * 9), lambda: kvq.paged_read(*[None] * 7, n_tokens=1),
             lambda: kvq.paged_attention_decode(*[None] * 7, sm_scale=1.0),
             lambda: kvq.paged_attention_prefill(*[None] * 8, sm_scale=1.0)):
    for _ in range(2):
        try:
            call()
        except ImportError as e:
            assert "_kvq_torch.so" in str(e)
        else:
            raise AssertionError("no ImportError")
"""


@pytest.mark.parametrize("torch_side", [None, b"", b"\x7fELF not a library"])
def test_codec_without_the_torch_side(tmp_path, torch_side):
    pkg = tmp_path / PKG
    pkg.mkdir()
    for name in ("__init__.py", "kvq.py", "workloads.py"):
        shutil.copy(os.path.join(ROOT, PKG, name), pkg / name)
    os.symlink(os.path.join(ROOT, PKG, "libkvq.so"), pkg / "libkvq.so")
    if torch_side is not None:
        (pkg / "_kvq_torch.so").write_bytes(torch_side)
    r = subprocess.run([sys.executable, "-c", CODE], cwd=tmp_path, capture_output=True, text=True, timeout=300,
                       env={k: v for k, v in os.environ.items() if k != "PYTHONPATH"})
    assert r.returncode == 0, r.stderr[-2000:]


def test_torch_side_is_loaded_by_the_first_paged_call():
    """Here, where it is built: refusals come from it."""
    from kv_cache_quantization_02_b200 import kvq
    with pytest.raises(ValueError, match="block_table must be a torch.Tensor"):
        kvq.paged_write(*[None] * 9)
