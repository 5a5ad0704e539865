"""CPU checks of the 8-bit cache's entry points: bad arguments are refused, with a
reason, before anything touches CUDA."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from heterogeneous_lora_gemm_gb300 import build as b
    b.build()
    from heterogeneous_lora_gemm_gb300 import mlora
    return mlora


OK = dict(k_codes=16, k_scale=16, v_codes=16, v_scale=16, n_pages=4, page_size=16, kv_heads=2, head_dim=64, q_heads=4,
          prompt_bytes=0)


@pytest.mark.parametrize("change,code", [
    (dict(k_codes=None), 1), (dict(v_codes=None), 1), (dict(k_scale=None), 1), (dict(v_scale=None), 1),
    (dict(k_codes=24), 1), (dict(v_codes=8), 1), (dict(k_scale=2), 1),
    (dict(n_pages=0), 1), (dict(kv_heads=0), 1), (dict(q_heads=0), 1), (dict(q_heads=5), 1), (dict(q_heads=65536), 1),
    (dict(page_size=8), 8), (dict(page_size=24), 8), (dict(page_size=272), 8), (dict(page_size=0), 8),
    (dict(head_dim=8), 8), (dict(head_dim=72), 8), (dict(head_dim=272), 8), (dict(head_dim=-16), 8),
    (dict(n_pages=1 << 27), 8),
])
def test_create_refuses(lib, change, code):
    h = ctypes.c_void_p(123)
    args = {**OK, **change}
    assert lib.lib().mlora_cache_create(*args.values(), ctypes.byref(h)) == code
    assert h.value is None and lib.last_error()


def test_null_cache_is_invalid_arg(lib):
    L = lib.lib()
    assert L.mlora_cache_create(16, 16, 16, 16, 4, 16, 2, 64, 4, 0, None) == 1
    for fn in (L.mlora_cache_append, L.mlora_cache_read):
        assert fn(None, 16, 64, 64, 16, 64, 64, 1, 1, None, 16, 16, 1, 1, 1, None) == 1
    assert L.mlora_cache_attend(None, 16, 64, 64, 16, 64, 64, 1, 1, None, 16, 16, 1, 1, 1, 1.0, 0, None) == 1
    assert L.mlora_cache_status(None, None) == 1
    assert L.mlora_cache_destroy(None) == 0


def test_step_status_has_a_text(lib):
    assert "out of range" in lib.status_string(lib.MLORA_ERR_DEVICE_STEP)
