"""The 8-bit cache's attention at the edges of what its calls accept: against 64 bits, with the
tolerances of test_gpu_cache.py unless a test says otherwise."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():   # pragma: no cover - CPU machine
    pytest.skip("needs a GPU", allow_module_level=True)

from heterogeneous_lora_gemm_gb300 import Cache, mlora  # noqa: E402
from test_gpu_cache import F, Setup, as_np, check_attend, offsets_of, plain_attend, strided  # noqa: E402


# ---- windows --------------------------------------------------------------- #
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths,H,G,D,ps", [
    ([7, 1, 6], [3, 90, 2], 2, 2, 64, 16),                # few rows, some at negative positions
    ([5, 3], [2, 700], 1, 1, 256, 32),
    ([6, 40], [2, 30], 2, 4, 128, 64),                    # prompts, left-padded
    ([300, 20], [7, 500], 1, 16, 128, 64),                # and converted ahead
])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 8, 2 ** 30])
def test_a_window_larger_than_any_position_is_no_window(rows, lengths, H, G, D, ps, window, dtype):
    u = Setup(lengths, H, D, ps, Hq=H * G, seed=40)
    limited = check_attend(u, rows, dtype, window)
    assert torch.equal(limited, check_attend(u, rows, dtype, 0))
