"""The compiled binding of the serving calls: the rest of the package does without it (CPU only)."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_and_attention_do_not_load_the_binding():
    code = ("import quantized_attention_int8_b200 as qa\n"
            "import torch\n"
            "assert qa.sage_workspace_bytes(1, 2, 2, 128, 64) > 0\n"
            "x = torch.zeros(1, 2, 8, 64, dtype=torch.float16)\n"
            "try:\n    qa.sage_attn(x, x, x)\nexcept ValueError:\n    pass\n"
            "assert '_sage_binding' not in open('/proc/self/maps').read()\n"
            "try:\n    qa.sage_qk_norm_rope(x, x)\nexcept ValueError:\n    pass\n"
            "assert '_sage_binding' in open('/proc/self/maps').read()\n")
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True)


def test_a_binding_of_another_torch_is_not_taken(lib, monkeypatch):
    assert torch.__version__ in os.path.basename(lib.BINDING_PATH) and os.path.exists(lib.BINDING_PATH)
    monkeypatch.setattr(lib, "_binding", None)
    monkeypatch.setattr(lib, "BINDING_PATH", lib.BINDING_PATH.replace(torch.__version__, "0.0.0"))
    x = torch.zeros(2, 4, 64, dtype=torch.float16)
    with pytest.raises(ImportError, match="not built"):
        lib.sage_qk_norm_rope(x, x)
