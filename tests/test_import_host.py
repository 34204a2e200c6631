"""The package without its native module for torch tensors (another Python or
torch than the one it was built for): what does not need it is there."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import sys

class Blocked:
    def find_spec(self, name, path=None, target=None):
        if name.endswith("_fp4_torch"):
            raise ImportError("undefined symbol: of another torch")

sys.meta_path.insert(0, Blocked())
import torch
import joint_video_audio_b200 as j
"""


def _run(code):
    r = subprocess.run([sys.executable, "-c", WITHOUT + code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_the_package_imports_and_its_block_works():
    out = _run("""
assert "joint_video_audio_b200._fp4_torch" not in sys.modules
import h3_inputs as hi
b = j.H3Block(hi.make_inputs("tiny_320").dims)
print(b.workspace_bytes(320) > 0, j.Model is not None, j.quantize_fp4.__name__)
""")
    assert out.split() == ["True", "True", "quantize_fp4"]


def test_a_4_bit_call_names_what_is_missing():
    out = _run("""
i = torch.zeros(4, dtype=torch.int32)
x = torch.zeros(4, 256, dtype=torch.bfloat16)
for call in (lambda: j.quantize_fp4(x), lambda: j.Fp4Tensor(4, 256), lambda: j.sandwich_norm(x, x, i, i, torch.zeros(1, 1, 6, 256))):
    try:
        call()
    except ImportError as e:
        print("_fp4_torch" in str(e) and "build.py" in str(e) and "undefined symbol" in str(e))
""")
    assert out.split() == ["True"] * 3


def test_the_module_is_imported_once():
    import joint_video_audio_b200 as j
    from joint_video_audio_b200 import fp4
    j.Fp4Tensor(4, 256, device="cpu")
    assert {"layout", "quantize", "dequantize", "gemm", "sandwich"} <= set(vars(fp4._host))
